// What the two directions of the block norm share on the host.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "launch.h"

namespace moe {
namespace blk {

constexpr int kMaxGroupThreads = 512;      // threads of a row's group, 8 * nch columns each
// Dynamic shared memory per CTA (227 KB with the kernels' own).
constexpr int kNormSmem = 224 * 1024 + 256;
// Rows staged per group, one or two (with three the gradient took 46.5 us, not
// 43.4, at 4,096 x 2,560).
constexpr int kMaxStages = 2;
constexpr int kMaxStagedChunks = 2;        // wider rows (H > 8192) are read without staging

// How a launch cuts its rows: CTAs of `groups` groups of `nt` threads, each
// group with `stages` rows of `stage` bytes in shared memory.
struct NormPlan {
  int nt, nch, groups, stages, stage, grid, smem;
  int gains;  // bytes of c1 and c2 behind the stages
  int64_t by[8];  // bytes from a group's row to its next, per operand
};

// slot: bytes per thread of all operands' eight columns; chunked: how
// many operands are staged by chunks at most (kByChunks); max_threads: threads
// per CTA where a thread has eight columns.  One CTA per SM walks the rows (more where
// CTAs are small): a row's two sums put two barriers between its reads and its
// writes, so the copies of the rows ahead, not more threads, keep the memory
// busy.
inline NormPlan norm_plan(int T, int H, int slot, int chunked, int max_threads) {
  NormPlan p;
  const int chunks = (H + 7) / 8;
  p.nch = chunks <= kMaxGroupThreads ? 1 : chunks <= 2 * kMaxGroupThreads ? 2 : 4;
  p.nt = ((chunks + p.nch - 1) / p.nch + 31) / 32 * 32;
  if (p.nch > 1) max_threads = kMaxGroupThreads;
  const int sms = sm_count();
  p.groups = std::max(1, std::min(p.nt == 32 ? 32 : 15, max_threads / p.nt));
  p.groups = std::max(1, std::min(p.groups, (T + sms - 1) / sms));
  p.stage = p.nch <= kMaxStagedChunks ? slot * p.nch * p.nt + 16 * chunked : 0;
  p.gains = p.nch <= kMaxStagedChunks ? 2 * 32 * p.nch * p.nt : 0;
  const int room = kNormSmem - p.gains;
  while (p.groups > 1 && p.stage * p.groups * 2 > room) --p.groups;
  p.stages = p.stage > 0 ? std::max(1, std::min(kMaxStages, room / (p.stage * p.groups))) : 1;
  const int per_sm = std::max(1, std::min(max_threads / (p.nt * p.groups),
                                          p.stage > 0 ? kNormSmem / (p.stage * p.groups * p.stages + p.gains) : 8));
  p.grid = std::max(1, std::min((T + p.groups - 1) / p.groups, sms * per_sm));
  const int rows = (T + p.grid * p.groups - 1) / (p.grid * p.groups);  // per group
  p.stages = std::max(1, std::min(p.stages, rows));
  p.smem = p.stage * p.groups * p.stages + p.gains;
  return p;
}

inline void plan_steps(NormPlan& p, std::initializer_list<Rows> all) {
  int i = 0;
  const int64_t step = static_cast<int64_t>(p.grid) * p.groups;
  for (const Rows& r : all) p.by[i++] = step * r.ld * (r.type == MOE_ROW_F32 ? 4 : 2);
}

// The widest unit of adjacent columns that the width and every row allow.
inline int norm_unit(int H, std::initializer_list<Rows> all) {
  int g = H % 4 == 0 ? 4 : H % 2 == 0 ? 2 : 1;
  for (const Rows& r : all)
    while (g > 1 && !starts_on(r, g)) g /= 2;
  return g;
}

// Raise a kernel's shared memory limit once per device.
template <typename K>
cudaError_t allow_smem(K kern, std::atomic<uint64_t>& done) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t r = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
  if (r == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return r;
}

// f(type tag of x, type tag of y, unit, chunks) with the numbers as integral
// constants.
template <typename F>
cudaError_t norm_dispatch(int xt, int yt, int unit, int nch, F&& f) {
  auto c = [&](auto tx, auto ty, auto g) {
    if (nch == 1) return f(tx, ty, g, std::integral_constant<int, 1>());
    if (nch == 2) return f(tx, ty, g, std::integral_constant<int, 2>());
    return f(tx, ty, g, std::integral_constant<int, 4>());
  };
  auto u = [&](auto tx, auto ty) {
    if (unit == 4) return c(tx, ty, std::integral_constant<int, 4>());
    if (unit == 2) return c(tx, ty, std::integral_constant<int, 2>());
    return c(tx, ty, std::integral_constant<int, 1>());
  };
  using B = uint16_t;
  if (xt == MOE_ROW_F32) return yt == MOE_ROW_F32 ? u(float(), float()) : u(float(), B());
  return yt == MOE_ROW_F32 ? u(B(), float()) : u(B(), B());
}

inline int row_bytes8(const Rows& r) { return r.p == nullptr ? 0 : r.type == MOE_ROW_F32 ? 32 : 16; }

}  // namespace blk
}  // namespace moe
