// Grouped int8 products (moe_grouped_linear_i8, moe_grouped_ffn_i8) on the
// integer matrix instructions of gfx950.
//
// Rows are int8 codes with one scale per row, expert matrices packed int8 codes
// with one scale per output channel; the sums are exact int32 and the scales
// multiply them in fp32.  Three kinds of products share two kernels:
//   kLinear  y = sx * sw * (xq . W)                                     -> bf16 or fp32
//   kGateUp  a = silu(sx sg (xq . Wg)) * (sx su (xq . Wu)), quantised per row and
//            128 columns (the columns of one tile)                      -> codes + scales
//   kDown    h = sw * sum over blocks of 128: sa[block] * (aq . Wd over the block)  -> bf16
// Quantising the SwiGLU product where it is made needs the largest magnitude of a
// row over the columns that share a scale, so a tile owns whole blocks: 128 columns.
// A scale for each 128 columns instead of one for the row keeps the product out of
// memory in 32 bits (N * I * 4 bytes written and read) and needs no launch in
// between; the price is one conversion and one fma per 128 products in kDown.
//
// v_mfma_i32_16x16x64_i8: lane 16 q + r holds the 16 codes K = 16 q .. 16 q + 15 of row
// r of either operand, which is what one KiB of a packed matrix holds in order.  The
// weight rows are the first operand, so in a 16x16 result lane 16 q + r has token
// row r and the output columns 4 q .. 4 q + 3.
#include <type_traits>

#include "common.h"
#include "item_plan.h"
#include "launch.h"
#include "quantize.h"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

enum Mode { kLinear, kGateUp, kDown };

constexpr int kBlock = 128;          // columns of the SwiGLU product that share a scale
constexpr int kStep = 64;            // K of one matrix instruction
constexpr int kMaxGroups = 2 * 512 + 256;

struct ProductArgs {
  const int8_t* a;         // codes of the rows: [n_x][K]; kDown: [n_rows][K]
  const float* as;         // their scales: [n_x]; kDown: [ceil(K / 128)][n_rows]
  const int8_t *w0, *w1;   // packed matrices [E+S][cols][K] (w1: up rows of kGateUp)
  const float *s0, *s1;    // channel scales [E+S][cols]
  const int* x_rows;       // row list (nullptr: sorted row n reads row n)
  const int* offs;
  void* out;               // [n_rows][cols]: values, kGateUp: codes
  float* out_scale;        // kGateUp: [ceil(cols / 128)][n_rows]
  int n_x, n_rows, K, cols;
  int G, E, nseg;
};

__device__ __forceinline__ int src_row(const ProductArgs& p, int n) {
  return p.x_rows ? min(max(p.x_rows[n], 0), p.n_x - 1) : n;
}

__device__ __forceinline__ i32x4 mfma_i8(const uint4& w, const uint4& x, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), c, 0, 0, 0);
}

// silu(g) * u; the hardware's exponential and reciprocal are within 2 ulp, far below
// half a code of the quantisation that follows
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

template <class Out>
__device__ __forceinline__ void store4(Out* p, const float (&v)[4]) {
  if constexpr (sizeof(Out) == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  else
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// ---- small groups: weights stream from HBM into the matrix operands ----------------
// One block of eight waves per item (at most 16 * MF rows of a group, 128 output
// columns): each wave owns 16 columns (kGateUp: 16 gate rows and 16 up rows) and
// reads their weights once; the rows' codes are staged through LDS, 512 of K at a
// time, double buffered, and shared by the waves.
constexpr int kThreadsS = 512;
constexpr int kWavesS = kThreadsS / kWave;
constexpr int kChunk = 512;
constexpr int kPitch = kChunk + 16;  // bytes of a staged row: 16 rows start in 16 different bank groups

// The block's item, found from the group offsets (every thread calls it).
__device__ Item find_item(const ProductArgs& p, int BM, int nch) {
  constexpr int GPT = (kMaxGroups + kThreadsS - 1) / kThreadsS;
  __shared__ int wsum[kWavesS];
  __shared__ Item found;
  const int tid = threadIdx.x, lane = lane_id(), w = tid >> 6;
  const int x = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
  if (tid == 0) found = Item{0, 0, 0, 0, 0, 0};
  GroupRows gr[GPT];
  int s = 0;
#pragma unroll
  for (int q = 0; q < GPT; ++q) {
    const int g = tid * GPT + q;
    gr[q] = GroupRows{0, 0, 0, 0, 0, 0};
    if (g < p.G) {
      gr[q] = group_rows(p.offs, p.n_rows, p.E, p.nseg, BM, g);
      s += group_items(gr[q], g, nch, x);
    }
  }
  int incl = s;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int y = __shfl_up(incl, o, kWave);
    if (lane >= o) incl += y;
  }
  if (lane == kWave - 1) wsum[w] = incl;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int i = 0; i < kWavesS; ++i) base += i < w ? wsum[i] : 0;
  int t = base + incl - s;
  if (slot >= t && slot < t + s) {
#pragma unroll
    for (int q = 0; q < GPT; ++q) {
      const int g = tid * GPT + q;
      if (g >= p.G) break;
      const int n = group_items(gr[q], g, nch, x);
      if (slot >= t && slot < t + n) found = group_item(gr[q], g, nch, x, slot - t, BM, p.E, p.nseg);
      t += n;
    }
  }
  __syncthreads();
  return found;
}

template <int MF, Mode M, class Out>
__global__ __launch_bounds__(kThreadsS, 4) void stream_i8(ProductArgs p) {
  constexpr int BM = 16 * MF;
  constexpr int NF = M == kGateUp ? 2 : 1;
  constexpr int U = kChunk / kStep;
  constexpr int VPR = kChunk / 16;                          // 16-byte pieces of a staged row
  constexpr int APT = BM * VPR / kThreadsS;                 // pieces per thread
  constexpr int BPC = kChunk / kBlock;                      // blocks of 128 in a chunk
  static_assert(BM * VPR % kThreadsS == 0, "whole pieces per thread");
  __shared__ __attribute__((aligned(16))) int8_t As[2][BM * kPitch];
  __shared__ float Ss[M == kDown ? 2 : 1][M == kDown ? BPC * BM : 1];
  __shared__ uint32_t amax[M == kGateUp ? kWavesS : 1][M == kGateUp ? BM : 1];

  const Item it = find_item(p, BM, (p.cols + kBlock - 1) / kBlock);
  if (it.rows == 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int l16 = lane & 15, q = lane >> 4;
  const int K = p.K, cols = p.cols;
  const int col0 = it.chunk * kBlock + wave * 16;
  const bool live = col0 < cols;                            // cols % 64 == 0: all 16 columns or none
  const size_t rb = static_cast<size_t>(it.expert) * cols + (live ? col0 : cols - 16);
  const int8_t* bp[NF];
  bp[0] = p.w0 + rb * K + lane * 16;
  if constexpr (NF == 2) bp[1] = p.w1 + rb * K + lane * 16;

  const int8_t* arow[APT];
  uint4 stage[APT];
  float sstage = 0.f;
#pragma unroll
  for (int s = 0; s < APT; ++s) {
    const int r = (threadIdx.x + s * kThreadsS) / VPR;
    arow[s] = r < it.rows ? p.a + static_cast<size_t>(M == kDown ? it.row(r) : src_row(p, it.row(r))) * K : nullptr;
  }
  auto load_a = [&](int c) {
#pragma unroll
    for (int s = 0; s < APT; ++s) {
      const int k = c * kChunk + (threadIdx.x + s * kThreadsS) % VPR * 16;
      stage[s] = arow[s] && k < K ? *reinterpret_cast<const uint4*>(arow[s] + k) : make_uint4(0, 0, 0, 0);
    }
    if constexpr (M == kDown) {
      const int r = threadIdx.x % BM, b = c * BPC + threadIdx.x / BM;
      sstage = threadIdx.x < BPC * BM && r < it.rows && b * kBlock < K
                   ? p.as[static_cast<size_t>(b) * p.n_rows + it.row(r)] : 0.f;
    }
  };
  auto store_a = [&](int buf) {
#pragma unroll
    for (int s = 0; s < APT; ++s) {
      const int i = threadIdx.x + s * kThreadsS;
      *reinterpret_cast<uint4*>(&As[buf][(i / VPR) * kPitch + (i % VPR) * 16]) = stage[s];
    }
    if constexpr (M == kDown)
      if (threadIdx.x < BPC * BM) Ss[buf][threadIdx.x] = sstage;
  };

  i32x4 acc[MF][NF];
  f32x4 facc[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    facc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  }
  const int nc = (K + kChunk - 1) / kChunk;
  load_a(0);
  store_a(0);
  for (int c = 0; c < nc; ++c) {
    uint4 b[U][NF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kk = c * kChunk + u * kStep;                // K % 64 == 0: whole steps
#pragma unroll
      for (int j = 0; j < NF; ++j)
        b[u][j] = kk < K ? *reinterpret_cast<const uint4*>(bp[j] + static_cast<size_t>(kk) * 16) : make_uint4(0, 0, 0, 0);
    }
    const bool more = c + 1 < nc;
    if (more) load_a(c + 1);
    __syncthreads();                                        // chunk c of the rows is staged
    const int8_t* as = As[c & 1] + l16 * kPitch + 16 * q;
    if constexpr (M == kDown) {
#pragma unroll
      for (int u = 0; u < U; u += 2)
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          const uint4 a0 = *reinterpret_cast<const uint4*>(as + 16 * i * kPitch + u * kStep);
          const uint4 a1 = *reinterpret_cast<const uint4*>(as + 16 * i * kPitch + (u + 1) * kStep);
          const i32x4 t = mfma_i8(b[u + 1][0], a1, mfma_i8(b[u][0], a0, i32x4{0, 0, 0, 0}));
          const float s = Ss[c & 1][(u / 2) * BM + 16 * i + l16];
#pragma unroll
          for (int r = 0; r < 4; ++r) facc[i][r] = __builtin_fmaf(static_cast<float>(t[r]), s, facc[i][r]);
        }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          const uint4 av = *reinterpret_cast<const uint4*>(as + 16 * i * kPitch + u * kStep);
#pragma unroll
          for (int j = 0; j < NF; ++j) acc[i][j] = mfma_i8(b[u][j], av, acc[i][j]);
        }
    }
    if (more) store_a((c + 1) & 1);                         // last read before this chunk's barrier
  }

  const int n = col0 + 4 * q;
  const size_t so = static_cast<size_t>(it.expert) * cols + (live ? n : 0);
  const f32x4 w0 = *reinterpret_cast<const f32x4*>(p.s0 + so);
  if constexpr (M == kGateUp) {
    const f32x4 w1 = *reinterpret_cast<const f32x4*>(p.s1 + so);
    float v[MF][4];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = 16 * i + l16;
      const float sx = m < it.rows ? p.as[src_row(p, it.row(m))] : 0.f;
      uint32_t big = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[i][r] = silu_mul(static_cast<float>(acc[i][0][r]) * (sx * w0[r]), static_cast<float>(acc[i][1][r]) * (sx * w1[r]));
        big = max(big, abs_bits(v[i][r]));
      }
      big = max(big, static_cast<uint32_t>(__shfl_xor(static_cast<int>(big), 16, kWave)));
      big = max(big, static_cast<uint32_t>(__shfl_xor(static_cast<int>(big), 32, kWave)));
      if (q == 0) amax[wave][m] = live ? big : 0u;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = 16 * i + l16;
      if (m >= it.rows) continue;
      uint32_t big = amax[0][m];
#pragma unroll
      for (int w = 1; w < kWavesS; ++w) big = max(big, amax[w][m]);
      const QuantScale qs = quant_scale(big);
      const int row = it.row(m);
      if (live)
        *reinterpret_cast<uint32_t*>(static_cast<int8_t*>(p.out) + static_cast<size_t>(row) * cols + n) =
            pack_codes(quant_code(v[i][0], qs), quant_code(v[i][1], qs), quant_code(v[i][2], qs), quant_code(v[i][3], qs));
      if (wave == 0 && q == 0) p.out_scale[static_cast<size_t>(it.chunk) * p.n_rows + row] = qs.scale;
    }
  } else {
    if (!live) return;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = 16 * i + l16;
      if (m >= it.rows) continue;
      const int row = it.row(m);
      float v[4];
      if constexpr (M == kDown) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = facc[i][r] * w0[r];
      } else {
        const float sx = p.as[src_row(p, row)];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = static_cast<float>(acc[i][0][r]) * (sx * w0[r]);
      }
      store4(static_cast<Out*>(p.out) + static_cast<size_t>(row) * cols + n, v);
    }
  }
}

int pick_mf(int avg) { return avg <= 12 ? 1 : avg <= 28 ? 2 : 4; }

template <Mode M, class Out>
void launch_product(const ProductArgs& p, hipStream_t stream) {
  const int avg = p.n_rows / p.G;
  const int mf = pick_mf(avg);
  const int max_tiles = (p.n_rows + 16 * mf - 1) / (16 * mf) + p.G;
  dim3 grid(item_grid(max_tiles, (p.cols + kBlock - 1) / kBlock)), block(kThreadsS);
  switch (mf) {
    case 1: hipLaunchKernelGGL((stream_i8<1, M, Out>), grid, block, 0, stream, p); break;
    case 2: hipLaunchKernelGGL((stream_i8<2, M, Out>), grid, block, 0, stream, p); break;
    default: hipLaunchKernelGGL((stream_i8<4, M, Out>), grid, block, 0, stream, p); break;
  }
}

ProductArgs product_args(const GroupedI8& g, int K, int cols) {
  ProductArgs p{};
  p.x_rows = g.x_rows;
  p.offs = g.group_offsets;
  p.n_x = g.n_x;
  p.n_rows = g.n_rows;
  p.K = K;
  p.cols = cols;
  p.G = g.nseg * g.E + g.n_shared;
  p.E = g.E;
  p.nseg = g.nseg;
  return p;
}

// Workspace of the FFN: token codes and scales, SwiGLU codes and block scales.
struct FfnI8Layout {
  size_t xs, aq, as, total;   // byte offsets (the token codes start at 0)
};
FfnI8Layout ffn_i8_layout(int n_rows, int n_tokens, int d, int I) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  FfnI8Layout L;
  L.xs = up(static_cast<size_t>(n_tokens) * d);
  L.aq = L.xs + up(static_cast<size_t>(n_tokens) * 4);
  L.as = L.aq + up(static_cast<size_t>(n_rows) * I);
  L.total = L.as + up(static_cast<size_t>((I + kBlock - 1) / kBlock) * n_rows * 4);
  return L;
}

}  // namespace

hipError_t launch_grouped_linear_i8(const GroupedI8& g, const int8_t* xq, const float* xs, int K, int O,
                                    const int8_t* w, const float* ws, int bf16, void* y, hipStream_t stream) {
  ProductArgs p = product_args(g, K, O);
  p.a = xq;
  p.as = xs;
  p.w0 = w;
  p.s0 = ws;
  p.out = y;
  if (bf16) launch_product<kLinear, uint16_t>(p, stream);
  else launch_product<kLinear, float>(p, stream);
  return hipGetLastError();
}

size_t ffn_i8_workspace_bytes(int n_rows, int n_tokens, int d, int I) {
  return ffn_i8_layout(n_rows, n_tokens, d, I).total;
}

hipError_t launch_ffn_i8(const FfnI8Args& a, void* workspace, hipStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  const FfnI8Layout L = ffn_i8_layout(a.g.n_rows, a.g.n_x, a.d, a.I);
  int8_t* xq = reinterpret_cast<int8_t*>(ws);
  float* xs = reinterpret_cast<float*>(ws + L.xs);
  const hipError_t e = launch_quantize_rows(a.x, 1, a.g.n_x, a.d, xq, xs, stream);
  if (e != hipSuccess) return e;
  ProductArgs p = product_args(a.g, a.d, a.I);
  p.a = xq;
  p.as = xs;
  p.w0 = a.w_gate;
  p.w1 = a.w_up;
  p.s0 = a.s_gate;
  p.s1 = a.s_up;
  p.out = ws + L.aq;
  p.out_scale = reinterpret_cast<float*>(ws + L.as);
  launch_product<kGateUp, int8_t>(p, stream);
  ProductArgs h = product_args(a.g, a.I, a.d);
  h.a = reinterpret_cast<const int8_t*>(ws + L.aq);
  h.as = p.out_scale;
  h.w0 = a.w_down;
  h.s0 = a.s_down;
  h.out = a.h_sorted;
  launch_product<kDown, uint16_t>(h, stream);
  return hipGetLastError();
}

}  // namespace moe
