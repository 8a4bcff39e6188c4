// Routing with scores (moe_route): softmax or sigmoid scores, a balance bias for
// the selection, groups of experts, top-k, scaled weights.  One wavefront per
// token; lane holds the experts 64 i + lane.
//
// Everything that decides an id is computed in double, so that neighbouring
// scores fall as the definition says.
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

__device__ __forceinline__ double wave_max_d(double v) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o, kWave));
  return v;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, size_t i) {
  float v;
  if constexpr (BF16) v = bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else v = static_cast<const float*>(p)[i];
  return v != v ? -__builtin_inff() : v;
}

template <int P, bool BF16>
__global__ __launch_bounds__(kWave * kWavesPerBlock) void route_kernel(const void* __restrict__ logits,
                                                                       const float* __restrict__ bias, RouteArgs a) {
  __shared__ double vals[kWavesPerBlock][P * kWave];
  const int w = threadIdx.x >> 6, lane = lane_id();
  const int t = blockIdx.x * kWavesPerBlock + w;
  if (t >= a.T) return;                         // whole waves leave, no block barrier below
  const int E = a.E;

  double l[P], s[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + i * kWave;
    l[i] = e < E ? static_cast<double>(load_logit<BF16>(logits, static_cast<size_t>(t) * E + e)) : -__builtin_inf();
  }
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = 1.0 / (1.0 + exp(-l[i]));
  } else {
    double m = l[0];
#pragma unroll
    for (int i = 1; i < P; ++i) m = fmax(m, l[i]);
    m = wave_max_d(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      // the largest logits count 1 also where they are +inf; an all -inf row counts nothing
      s[i] = l[i] == -__builtin_inf() ? 0.0 : (l[i] == m ? 1.0 : exp(l[i] - m));
      sum += s[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  }

  uint64_t key[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + i * kWave;
    const double c = bias && e < E ? s[i] + static_cast<double>(bias[e]) : l[i];
    key[i] = e < E ? key_of(c) : 0ull;
    if (e < E && a.n_groups > 1) vals[w][e] = (bias || !a.top2) ? c : s[i];
  }

  if (a.n_groups > 1) {
    // the wave's own values, through LDS: its writes before its reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // value of group `lane` (n_groups <= 64)
    const int size = E / a.n_groups;
    double v1 = -__builtin_inf(), v2 = -__builtin_inf();
    if (lane < a.n_groups) {
      for (int j = 0; j < size; ++j) {
        double v = vals[w][lane * size + j];
        if (v != v) v = -__builtin_inf();
        v2 = fmax(v2, fmin(v1, v));
        v1 = fmax(v1, v);
      }
    }
    const uint64_t gk = lane < a.n_groups ? key_of(a.top2 && size > 1 ? v1 + v2 : v1) : 0ull;
    int rank = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      const uint64_t o = __shfl(gk, g, kWave);
      rank += (o > gk || (o == gk && g < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.n_groups && rank < a.top_groups);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int g = (lane + i * kWave) / size;
      if (g >= a.n_groups || !((kept >> g) & 1)) key[i] = 0ull;
    }
  }

  // k rounds: the largest key, the lowest expert that has it; round r is kept by lane r % 64, slot r / 64
  double cs[P];
  int cid[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    cs[i] = 0.0;
    cid[i] = 0;
  }
  for (int r = 0; r < a.k; ++r) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < P; ++i) best = key[i] > best ? key[i] : best;
    const uint64_t win = wave_max_u64(best);
    int wi = 0, wl = 0;
    double ws = 0.0;
#pragma unroll
    for (int i = P - 1; i >= 0; --i) {
      const uint64_t m = __ballot(key[i] == win);
      if (m) {
        wi = i;
        wl = __ffsll(static_cast<unsigned long long>(m)) - 1;
        ws = s[i];
      }
    }
    ws = __shfl(ws, wl, kWave);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (i == wi && lane == wl) key[i] = 0ull;
      if (r == i * kWave + lane) {
        cs[i] = ws;
        cid[i] = wi * kWave + wl;
      }
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) sum += cs[i];
  const double denom = a.renormalize ? wave_sum(sum) : 1.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int slot = i * kWave + lane;
    if (slot < a.k) {
      a.topk_ids[static_cast<size_t>(t) * a.k + slot] = cid[i];
      a.topk_w[static_cast<size_t>(t) * a.k + slot] =
          denom > 0.0 ? static_cast<float>(cs[i] / denom * static_cast<double>(a.scale)) : 0.0f;
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

hipError_t launch_route(const void* logits, const float* bias, const RouteArgs& a, hipStream_t stream) {
  if (a.E <= 64) launch_p<1>(logits, bias, a, stream);
  else if (a.E <= 128) launch_p<2>(logits, bias, a, stream);
  else if (a.E <= 256) launch_p<4>(logits, bias, a, stream);
  else launch_p<8>(logits, bias, a, stream);
  return hipGetLastError();
}

}  // namespace moe
