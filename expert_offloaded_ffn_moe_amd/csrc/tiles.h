// What the tiled products of 8-bit codes share: the tiles' order, the choice among them, and loads from
// memory to LDS with the waits that count them.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {
namespace {

typedef __attribute__((address_space(3))) void lvoid;

// Workgroups are dealt to the 8 XCDs round-robin; each XCD gets one contiguous range of
// the tiles, so that the tiles of its L2 share rows and channels.
__device__ __forceinline__ int xcd_order(int b, int nb) {
  constexpr int kXcd = 8;
  const int per = nb / kXcd, rem = nb % kXcd, x = b % kXcd, i = b / kXcd;
  return x < rem ? x * (per + 1) + i : rem * (per + 1) + (x - rem) * per + i;
}

// All but the newest N of this wave's loads are in, every LDS read too, and so it is for every
// wave of the workgroup. One block: what follows reads LDS that other waves' loads wrote.
template <int N>
__device__ __forceinline__ void meet_with_loads_but() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes from each lane's address to LDS at `to` + 16 lane. Written as one block, so that
// the compiler, which cannot tell the ring's buffers apart, adds no wait for it before the
// LDS reads of the others: meet_with_loads_but counts these loads instead. It has no output
// register. (A write of M0 is followed by one wait state before its use.)
__device__ __forceinline__ void load_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory", "m0");
}
// 4 bytes from each lane's address to LDS at `to` + 4 lane.
__device__ __forceinline__ void load_one_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "memory", "m0");
}

// A tile, and what a step of K costs a CU in it.
struct Tile {
  int tokens, channels;
  float cost;
};
constexpr int kCus = 256;

// The tile, from `first` on, whose rounds over the CUs cost least.
template <int COUNT>
int choose_tile(const Tile (&tiles)[COUNT], int64_t T, int64_t channels, int first = 0) {
  int best = first;
  float least = 0.f;
  for (int i = first; i < COUNT; ++i) {
    const int64_t n = ((T - 1) / tiles[i].tokens + 1) * ((channels - 1) / tiles[i].channels + 1);
    const float cost = (float)((n - 1) / kCus + 1) * tiles[i].cost;
    if (i == first || cost < least) {
      best = i;
      least = cost;
    }
  }
  return best;
}

}  // namespace
}  // namespace moe
