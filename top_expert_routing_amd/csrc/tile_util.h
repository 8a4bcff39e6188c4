// Steps that the grouped products on int8 and FP8 codes share: exchanges between lanes, a block's
// work item, LDS-DMA loads and their waits.
#pragma once

#include "common.h"
#include "i8_plan.h"

// Lambdas over the kernel's state: a call that is not inlined would put that state in memory.
#define MOE_INLINE __attribute__((always_inline))

namespace moe {

// Exchanges over the four 16-lane rows q of a wave, on gfx950's row swaps; every lane takes part.
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {   // lanes 32-63 of a with lanes 0-31 of b
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0], b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {   // rows 1, 3 of a with rows 0, 2 of b
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0], b = r[1];
}
// d[j] of row q becomes d[q] of row j.
__device__ __forceinline__ void transpose_rows(uint32_t (&d)[4]) {
  swap32(d[0], d[2]);
  swap32(d[1], d[3]);
  swap16(d[0], d[1]);
  swap16(d[2], d[3]);
}

// silu(g) * u.  In half steps of 2^-24: g and u arrive within 3 each; exp(-g) is within
// 3 |g| (of g) + 1.3 |g| (the rounded argument of the exponential and its constant) + 4 (2 ulp), which
// counts in full where g is far below zero and by at most |g| e^-g / (1 + e^-g) < 0.28 above; the sum,
// the reciprocal (2 ulp) and the two products add 7.  Below g = -87 the reciprocal can flush to 0.
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

__device__ __forceinline__ uint32_t max_over_q(uint32_t m) {        // over the four lanes of a row
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16, kWave)));
  return max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32, kWave)));
}

// Sum of v over the lanes up to this one.
__device__ __forceinline__ int wave_prefix(int v) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int y = __shfl_up(v, o, kWave);
    if (lane_id() >= o) v += y;
  }
  return v;
}

// The block's item of a launch_of grid, found from the group offsets (Args: offs, n_rows, G, E, nseg).  Every wave finds it by itself, so that
// nothing waits for another: a lane counts the items of `per` neighbouring groups, a sum
// over the lanes tells whose the block's is, and where per > 1 the lanes then take that
// lane's groups one each.  The result is wave-uniform, in scalar registers.
template <class Args>
__device__ Item find_item(const Args& p, int BM, int nch) {
  const int block = blockIdx.y * i8::kMostX + blockIdx.x;    // launch_of
  const int lane = lane_id(), x = block % kXcds;
  const int per = (p.G + kWave - 1) / kWave;                // <= 64: at most 1280 groups
  int slot = block / kXcds;
  GroupRows r{0, 0, 0, 0, 0, 0};
  int n = 0, g0 = 0;
  for (int i = 0; i < per; ++i) {
    const int g = lane * per + i;
    if (g < p.G) {
      r = group_rows(p.offs, p.n_rows, p.E, p.nseg, BM, g);
      n += group_items(r, g, nch, x);
    }
  }
  int at = wave_prefix(n) - n;
  uint64_t here = __ballot(slot >= at && slot < at + n);
  if (here == 0) return Item{0, 0, 0, 0, 0, 0};
  int w = __builtin_ctzll(here);
  slot -= __builtin_amdgcn_readlane(at, w);
  if (per > 1) {
    g0 = w * per;
    n = 0;
    if (lane < per && g0 + lane < p.G) {
      r = group_rows(p.offs, p.n_rows, p.E, p.nseg, BM, g0 + lane);
      n = group_items(r, g0 + lane, nch, x);
    }
    at = wave_prefix(n) - n;
    here = __ballot(slot >= at && slot < at + n);
    w = __builtin_ctzll(here);
    slot -= __builtin_amdgcn_readlane(at, w);
  }
  const GroupRows u{__builtin_amdgcn_readlane(r.a0, w), __builtin_amdgcn_readlane(r.na, w),
                    __builtin_amdgcn_readlane(r.b0, w), __builtin_amdgcn_readlane(r.nb, w),
                    __builtin_amdgcn_readlane(r.t0, w), __builtin_amdgcn_readlane(r.nt, w)};
  return group_item(u, g0 + w, nch, x, slot, BM, p.E, p.nseg);
}

// LDS-DMA loads: each lane's 16 or 4 bytes go to LDS address lds + 16 (or 4) * lane.
// Inline assembly, so that the compiler does not wait for them before every LDS
// read; the waits are explicit.  M0 holds the LDS base; s_nop as below.
__device__ __forceinline__ void dma16(const void* g, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(g), "{m0}"(lds) : "memory");
}
// The same from a wave-uniform address plus a lane's 32-bit offset.  The address may have
// been put into its scalar registers by a vector instruction (a readfirstlane, or a
// v_readlane from the register a spilled scalar is kept in) just before; a vector memory
// instruction may use it five wait states later, and the compiler does not look for that
// hazard inside inline assembly: s_nop 4.
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint64_t u = static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32))) << 32 |
                     static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b)));
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(u), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void dma4(const void* g, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, off" : : "v"(g), "{m0}"(lds) : "memory");
}
// The same for the lanes of `mask`, from a wave-uniform address plus a lane's 32-bit offset or a lane's
// address.  Every lane of the wave takes part.
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds, uint64_t mask) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint64_t u = static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32))) << 32 |
                     static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b)));
  asm volatile("s_nop 4\n\ts_mov_b64 exec, %2\n\tglobal_load_lds_dword %0, %1\n\ts_mov_b64 exec, -1"
               : : "v"(off), "s"(u), "s"(mask), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void dma4(const void* g, uint32_t lds, uint64_t mask) {
  asm volatile("s_nop 4\n\ts_mov_b64 exec, %1\n\tglobal_load_lds_dword %0, off\n\ts_mov_b64 exec, -1"
               : : "v"(g), "s"(mask), "{m0}"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" : : "n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" : : : "memory"); }
// LDS writes of all waves before LDS reads of all waves, DMA loads left in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
  typedef __attribute__((address_space(3))) const uint8_t lds_byte;
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_byte*)p));
}

__device__ __forceinline__ Item uniform(const Item& i) {
  return Item{__builtin_amdgcn_readfirstlane(i.row0),   __builtin_amdgcn_readfirstlane(i.rows),
              __builtin_amdgcn_readfirstlane(i.expert), __builtin_amdgcn_readfirstlane(i.chunk),
              __builtin_amdgcn_readfirstlane(i.split),  __builtin_amdgcn_readfirstlane(i.row1)};
}

// CUs of the current device.
inline int device_cus() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    return 256;
  return cus;
}

}  // namespace moe
