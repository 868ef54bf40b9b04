// slots.h — the plan's slots as the experts' products walk them, and the
// pieces those kernels share: copies into LDS and the waits that order them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mb_internal.h"
#include "wave.h"

namespace mb {

constexpr int kExpertThreads = 256;
constexpr int kMaxPlanSlots = kMaxExperts + kMaxRanks * kMaxSlots;
constexpr int kTileN = 256;
constexpr int kCus = 256, kXcds = 8;
constexpr int kGroupM = 4;  // row tiles whose columns are walked together

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

typedef const __attribute__((address_space(4))) int32_t* plan_ptr;

// Rows [lo, hi) of slot j (r = j / NS), absolute in the buffer, and its
// expert; empty when it holds none. Only a broken plan needs the clamps.
template <class Args>
__device__ __forceinline__ void slot_rows(const Args& p, int j, int& lo, int& hi, int& e) {
  const int r = j / p.NS, i = j - r * p.NS;
  // the plan does not change under the kernel: constant memory
  auto cu = (plan_ptr)(p.cu + (size_t)r * (p.NS + 1) + i);
  lo = min(max(cu[0], 0), p.cap);
  hi = min(max(cu[1], lo), p.cap);
  e = i < p.Eh ? r * p.Eh + i : ((plan_ptr)p.rep)[(size_t)r * p.R + i - p.Eh];
  if ((unsigned)e >= (unsigned)p.E) hi = lo;
  lo += r * p.cap;
  hi += r * p.cap;
}

// first[j] = row tiles of the slots before j, first[nslots] = all of them.
template <int BM, class Args>
__device__ void tile_table(const Args& p, int nslots, int* first, int* part) {
  const int per = (nslots + kExpertThreads - 1) / kExpertThreads;
  const int j0 = threadIdx.x * per;
  int sum = 0;
  for (int j = j0; j < min(j0 + per, nslots); ++j) {
    int lo, hi, e;
    slot_rows(p, j, lo, hi, e);
    sum += (hi - lo + BM - 1) / BM;
  }
  const int incl = wave_inclusive_sum(sum);
  if ((threadIdx.x & 63) == 63) part[threadIdx.x >> 6] = incl;
  __syncthreads();
  int base = incl - sum;
  for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) base += part[i];
  for (int j = j0; j < min(j0 + per, nslots); ++j) {
    int lo, hi, e;
    slot_rows(p, j, lo, hi, e);
    first[j] = base;
    base += (hi - lo + BM - 1) / BM;
  }
  if (threadIdx.x == kExpertThreads - 1) first[nslots] = base;
  __syncthreads();
}

// The slot whose tiles hold row tile t.
__device__ __forceinline__ int slot_of(const int* first, int nslots, int t) {
  int lo = 0, hi = nslots;  // first[lo] <= t < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= t) lo = mid;
    else hi = mid;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

__device__ __forceinline__ i32x4 load16(const void* p) {
  return *static_cast<const i32x4*>(__builtin_assume_aligned(p, 16));
}

// Waits until this wave's LDS reads are done, then for the other waves.
__device__ __forceinline__ void read_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Waits until this wave's LDS reads are done and at most N of its memory
// operations (copies to LDS, stores) are outstanding, oldest first, then for
// the other waves.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

typedef __attribute__((address_space(3))) void* lds_ptr;

// Buffer descriptor of `bytes` bytes at p (wave-uniform). A read at voff +
// soff gives 0 where voff >= bytes - soff: soff must be below bytes, so what
// may pass the end is always in voff.
__device__ __forceinline__ i32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return i32x4{__builtin_amdgcn_readfirstlane((int)at),
               __builtin_amdgcn_readfirstlane((int)(at >> 32) & 0xffff),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// Copies 64 lanes' 16 bytes at buf[voff + soff] to consecutive places of LDS
// from `to` (wave-uniform; the instruction takes it from m0, one instruction
// after m0 was written). No register is written. In assembly because the
// compiler, for its builtin, waits for every copy in flight before the next
// read of any LDS; the waits that order copies and reads are wait_barrier's.
// The compiler does not look into the assembly for hazards: a scalar register
// that a vector instruction wrote (a lane read back, of a value or of a
// spilled register) is valid for memory instructions five wait states later.
// kNops waits that long before the copy (one now and then; where there are
// many, their buffer waits for all of them, see settled).
template <int kNops = 4>
__device__ __forceinline__ void copy16(i32x4 buf, lds_ptr to, uint32_t voff, uint32_t soff) {
  asm volatile("s_nop %4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               ::"{m0}"((uint32_t)(uintptr_t)to), "v"(voff), "s"(buf), "s"(soff), "n"(kNops)
               : "memory");
}

// For copies without that wait (copy16<0>): a buffer that has waited. Nothing
// of theirs may be read back from a vector register close before them, which
// the disassembled library is tested for.
__device__ __forceinline__ i32x4 settled(i32x4 buf) {
  asm volatile("s_nop 4" : "+s"(buf));
  return buf;
}

}  // namespace mb
