// The warp intrinsics of the row planner on the CPU: 32 lanes as ucontext fibers
// on one thread, switched round-robin at every warp exchange.  run_warp runs a
// function on all 32 lanes.
#pragma once

#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#define __device__
#define __forceinline__ inline
#define __host__
using std::min;

struct LaneIndex {
  unsigned x;
};
LaneIndex threadIdx;  // the running lane (set on every switch)

// 32 lanes as fibers.  A lane that reaches a barrier passes control to the
// next lane; the 32nd to arrive goes on, and the others resume in turn at their
// next switch, so every lane runs the code between two barriers once.
ucontext_t g_main, g_lane_ctx[32];
int g_arrived = 0;
bool g_finished[32];

void switch_to(int from, int to) {
  threadIdx.x = static_cast<unsigned>(to);
  swapcontext(&g_lane_ctx[from], &g_lane_ctx[to]);
  threadIdx.x = static_cast<unsigned>(from);
}

struct LaneBarrier {
  void wait() {
    const int lane = threadIdx.x & 31;
    if (++g_arrived == 32) {
      g_arrived = 0;
      return;
    }
    switch_to(lane, (lane + 1) & 31);
  }
};
LaneBarrier g_bar;
uint64_t g_slot[32];

// Every lane publishes v; each receives lane src's value.
template <class T>
T lane_exchange(T v, int src) {
  const int lane = threadIdx.x & 31;
  uint64_t bits = 0;
  std::memcpy(&bits, &v, sizeof(T));
  g_slot[lane] = bits;
  g_bar.wait();
  T r;
  std::memcpy(&r, &g_slot[src], sizeof(T));
  g_bar.wait();
  return r;
}
template <class T>
T __shfl_xor_sync(unsigned, T v, int o) {
  return lane_exchange(v, (threadIdx.x & 31) ^ o);
}
template <class T>
T __shfl_up_sync(unsigned, T v, int o) {
  const int lane = threadIdx.x & 31;
  return lane_exchange(v, lane >= o ? lane - o : lane);
}
template <class T>
T __shfl_sync(unsigned, T v, int src) {
  return lane_exchange(v, src);
}
unsigned __ballot_sync(unsigned, int pred) {
  const int lane = threadIdx.x & 31;
  g_slot[lane] = pred ? 1u : 0u;
  g_bar.wait();
  unsigned m = 0;
  for (int i = 0; i < 32; ++i)
    if (g_slot[i]) m |= 1u << i;
  g_bar.wait();
  return m;
}
int __any_sync(unsigned mask, int pred) { return __ballot_sync(mask, pred) != 0; }
int __ffs(unsigned x) { return __builtin_ffs(static_cast<int>(x)); }
template <class T>
T __ldg(const T *p) {
  return *p;
}

void (*g_warp_fn)(void *);
void *g_warp_arg;

void warp_lane_entry(int lane) {
  g_warp_fn(g_warp_arg);
  g_finished[lane] = true;
}

void run_warp(void (*fn)(void *), void *arg) {
  static std::vector<std::vector<char>> stacks(32, std::vector<char>(1 << 18));
  g_warp_fn = fn;
  g_warp_arg = arg;
  g_arrived = 0;
  for (int lane = 0; lane < 32; ++lane) {
    g_finished[lane] = false;
    getcontext(&g_lane_ctx[lane]);
    g_lane_ctx[lane].uc_stack.ss_sp = stacks[lane].data();
    g_lane_ctx[lane].uc_stack.ss_size = stacks[lane].size();
    g_lane_ctx[lane].uc_link = &g_main;
    makecontext(&g_lane_ctx[lane], reinterpret_cast<void (*)()>(warp_lane_entry), 1, lane);
  }
  // Lane 0 starts; control comes back whenever a lane returns, and the lanes
  // parked behind their last exchange are then run to their end.
  for (int round = 0; round < 33; ++round) {
    int lane = 0;
    while (lane < 32 && g_finished[lane]) ++lane;
    if (lane == 32) return;
    threadIdx.x = static_cast<unsigned>(lane);
    swapcontext(&g_main, &g_lane_ctx[lane]);
  }
  fprintf(stderr, "a lane did not finish\n");
  exit(1);
}
