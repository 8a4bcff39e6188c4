// Routing with scores (moe_route): softmax or sigmoid scores, a balance bias for
// the selection, groups of experts, top-k, scaled weights.  One wavefront per
// token; lane l holds the P experts l * P .. l * P + P - 1 (one 4 * P or 2 * P
// byte run of the row).
//
// Bound by the vector instructions: a token of 256 experts in 8 groups with a bias
// (k = 8, sigmoid) issues 642 and 238 scalar ones, so 8192 tokens, eight wavefronts a
// SIMD, need 8.5 us of the 11.0 measured; 16 tokens take 4.3 us, most of it the launch.
//   * Everything that decides an id is computed in double, so that neighbouring
//     scores fall as the definition says; fp64 runs at the fp32 rate here, and a
//     score (an exponential and a division) costs about 45 instructions a lane.
//   * Cross-lane steps stay in the vector registers (DPP).  A choice value is held as an
//     order-preserving 64-bit key; the maximum over the lanes is taken over the upper
//     halves, and over the lower ones only where several experts share the upper one.
//   * A round costs 18 vector instructions at P = 4: the masks of the lanes that hold the
//     maximum retire it and leave its rank in the key's place, so nothing is moved to
//     other lanes; each lane stores its chosen experts itself.  (Rounds that keep their
//     winner in lane r and gather its score afterwards: 12.9 us and, bf16, 4159 tokens of
//     160 experts, 11.0; now 8.7.)
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

// Monotone map of a double to uint64; NaN as -inf, -0 as +0.  The upper half of
// every key it returns is above kNoKey; smaller ones mark experts that cannot be
// chosen (any more).
constexpr uint32_t kNoKey = 0xffffeu;             // (the key of -inf is 0xfffff ffffffff)
__device__ __forceinline__ uint64_t key_of(double v) {
  v = v != v ? -__builtin_inf() : v + 0.0;
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t hi = static_cast<uint32_t>(u >> 32), sign = static_cast<uint32_t>(static_cast<int32_t>(hi) >> 31);
  return static_cast<uint64_t>(hi ^ (sign | 0x80000000u)) << 32 | (static_cast<uint32_t>(u) ^ sign);
}

// Lane l's value from the lane that CTRL names for it; 0 in the 16-lane rows that ROWS leaves out.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, static_cast<uint64_t>(dpp<CTRL, ROWS>(static_cast<uint32_t>(u >> 32))) << 32 |
                                        dpp<CTRL, ROWS>(static_cast<uint32_t>(u)));
}
constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;   // within a row: after all four, of 16 lanes
constexpr int kNextRow = 0x142, kUpperRows = 0x143;   // a row's last lane to the next row (rows 1, 3), lane 31's to rows 2, 3

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
  v = max(v, dpp<kNextRow, 0xa>(v));
  v = max(v, dpp<kUpperRows, 0xc>(v));
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
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
  v += dpp<kNextRow, 0xa>(v);
  v += dpp<kUpperRows, 0xc>(v);
  return lane_d(v, 63);
}

// The two largest of an ordered pair and a value, and of two ordered pairs.
__device__ __forceinline__ void push2(double& v1, double& v2, double o) {
  v2 = fmax(v2, fmin(v1, o));
  v1 = fmax(v1, o);
}
__device__ __forceinline__ void merge2(double& v1, double& v2, double o1, double o2) {
  v2 = fmax(fmin(v1, o1), fmax(v2, o2));
  v1 = fmax(v1, o1);
}

// Eight wavefronts a SIMD up to P = 4 (its 8192 tokens run at once), registers permitting above.
template <int P, bool BF16>
__global__ __launch_bounds__(kWave * kWavesPerBlock, P <= 4 ? 8 : P <= 6 ? 6 : 5) void route_kernel(const void* __restrict__ logits,
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
  } else if (e0 < E) {
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
    // far below zero 1 + exp(-l) leaves the doubles and exp(l) is the score to its last bit
    bool low = false;
#pragma unroll
    for (int i = 0; i < P; ++i) low |= l[i] < -700.0f && l[i] > -__builtin_inff();
    if (__any(low)) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (l[i] < -700.0f) s[i] = exp(static_cast<double>(l[i]));
    }
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
    const double share = sum > 0.0 ? 1.0 / sum : 0.0;        // the sum is at least 1 or 0
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] *= share;
  }

  uint32_t hi[P], lo[P];                        // choice values' keys
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint64_t key = key_of(bias ? s[i] + static_cast<double>(b[i]) : static_cast<double>(l[i]));
    hi[i] = e0 + i < E ? static_cast<uint32_t>(key >> 32) : 0u;
    lo[i] = static_cast<uint32_t>(key);
  }

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
    if (L > 0 && two) {
#pragma unroll
      for (int i = 0; i < P; ++i) push2(v1, v2, g[i]);
      // after each step every lane of the doubled run holds the run's two largest
      if (L > 1) merge2(v1, v2, dpp<kXor1>(v1), dpp<kXor1>(v2));
      if (L > 2) merge2(v1, v2, dpp<kXor2>(v1), dpp<kXor2>(v2));
      if (L > 4) merge2(v1, v2, dpp<kHalfMirror>(v1), dpp<kHalfMirror>(v2));
      if (L > 8) merge2(v1, v2, dpp<kMirror>(v1), dpp<kMirror>(v2));
      if (L > 16) merge2(v1, v2, __shfl_xor(v1, 16, kWave), __shfl_xor(v2, 16, kWave));
    } else if (L > 0) {
#pragma unroll
      for (int i = 0; i < P; ++i) v1 = fmax(v1, g[i]);
      if (L > 1) v1 = fmax(v1, dpp<kXor1>(v1));
      if (L > 2) v1 = fmax(v1, dpp<kXor2>(v1));
      if (L > 4) v1 = fmax(v1, dpp<kHalfMirror>(v1));
      if (L > 8) v1 = fmax(v1, dpp<kMirror>(v1));
      if (L > 16) v1 = fmax(v1, __shfl_xor(v1, 16, kWave));
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) vals[w][e0 + i] = g[i];
      // the wave's own values: its writes before its reads
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (lane < a.n_groups)
        for (int j = 0; j < size; ++j) push2(v1, v2, vals[w][lane * size + j]);
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
      for (int i = 0; i < P; ++i) hi[i] = stays ? hi[i] : 0u;
    } else {
      const uint64_t kept = __ballot(stays && lane < a.n_groups);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int gi = (e0 + i) / size;
        if (gi >= a.n_groups || !((kept >> gi) & 1)) hi[i] = 0u;
      }
    }
  }

  // k rounds: the largest key, the lowest expert that has it.  The expert chosen in round r
  // keeps r + 1 in place of its key's upper half (k <= 512, below kNoKey).  One expert nearly
  // always has the largest upper half alone; then its mask is all that the round needs.
  bool twice = false;                           // two experts of a lane share an upper half
#pragma unroll
  for (int i = 1; i < P; ++i)
#pragma unroll
    for (int j = 0; j < i; ++j) twice |= hi[i] == hi[j] && hi[i] > kNoKey;
  const bool pairs = __builtin_amdgcn_readfirstlane(__any(twice));
  for (int r = 1; r <= a.k; ++r) {
    uint32_t best = hi[0];
#pragma unroll
    for (int i = 1; i < P; ++i) best = max(best, hi[i]);
    const uint32_t top = wave_max_u32(best);
    uint64_t m[P], any = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      m[i] = __ballot(hi[i] == top);
      any |= m[i];
    }
    int n = __popcll(any);
    if (pairs) {
      n = 0;
#pragma unroll
      for (int i = 0; i < P; ++i) n += __popcll(m[i]);
    }
    if (n > 1) {                                // the lower halves tell, then the lowest lane and its lowest slot
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
      uint64_t left = any & -any;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        m[i] &= left;
        left &= ~m[i];
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) hi[i] = __builtin_amdgcn_inverse_ballot_w64(m[i]) ? static_cast<uint32_t>(r) : hi[i];
  }
  auto sum_chosen = [&]() {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) sum += hi[i] - 1u < static_cast<uint32_t>(a.k) ? s[i] : 0.0;
    return wave_sum_d(sum);
  };
  double denom = a.renormalize ? sum_chosen() : 1.0;
  if (denom > 0.0 && denom < 0x1p-700) {        // wave-uniform
    // Scores this small lose bits (below 2^-1022) and scale / denom can leave the doubles, but their
    // quotients are those of the exponentials of the logits, here taken relative to the largest chosen one
    // (all are finite: a sum of scores with an infinite logit is 0 or not small).
    float z[P], m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < P; ++i) {
      z[i] = -__builtin_inff();
      if (hi[i] - 1u < static_cast<uint32_t>(a.k)) {
        if constexpr (BF16) z[i] = bf16_to_f32(row[i]);
        else z[i] = row[i];
        if (z[i] != z[i]) z[i] = -__builtin_inff();
      }
      m = fmaxf(m, z[i]);
    }
    m = wave_max_f(m);
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = exp(static_cast<double>(z[i]) - static_cast<double>(m));
    denom = sum_chosen();
  }
  const double factor = denom > 0.0 ? static_cast<double>(a.scale) / denom : 0.0;
  // each lane writes its chosen experts at their places
  const size_t at = static_cast<size_t>(t) * a.k;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint32_t r = hi[i] - 1u;
    if (r < static_cast<uint32_t>(a.k)) {
      a.topk_ids[at + r] = e0 + i;
      a.topk_w[at + r] = static_cast<float>(s[i] * factor);
    }
  }
}

template <int P>
void launch_p(const void* logits, const float* bias, const RouteArgs& a, hipStream_t stream) {
  dim3 grid((a.T + kWavesPerBlock - 1) / kWavesPerBlock), block(kWave * kWavesPerBlock);
  if (a.bf16)
    hipLaunchKernelGGL((route_kernel<P, true>), grid, block, 0, stream, logits, bias, a);
  else
    hipLaunchKernelGGL((route_kernel<P, false>), grid, block, 0, stream, logits, bias, a);
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
