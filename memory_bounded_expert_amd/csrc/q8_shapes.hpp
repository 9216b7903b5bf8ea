// How rows in 8 bits are divided into launches.  Host only, no HIP.
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {

constexpr int kQ8GroupThreads = 256, kQ8GroupBlocks = 32;  // of a work-group: eight threads a block of 128 columns

// A launch of `rows` rows: `units` blocks in `groups` work-groups, with u / blocks = u magic
// >> shift for every u below units.
struct Q8Launch {
  int64_t rows;
  uint32_t units, groups, magic, shift;
};

// The next launch where `left` rows of `blocks` blocks are left.  A launch has fewer than
// 2^32 threads (HIP refuses others), so its units stay below 2^29.
inline Q8Launch q8_launch(int64_t left, int blocks) {
  constexpr int64_t kMostGroups = (((int64_t)1 << 32) - 1) / kQ8GroupThreads;
  Q8Launch l{};
  l.rows = std::min(left, kMostGroups * kQ8GroupBlocks / blocks);
  l.units = (uint32_t)(l.rows * blocks);
  l.groups = (l.units + kQ8GroupBlocks - 1) / kQ8GroupBlocks;
  // magic = ceil(2^shift / blocks), whose error, below blocks, times u stays below
  // 2^shift = 2^31 times a power of two >= blocks
  l.shift = 31;
  while ((1u << (l.shift - 31)) < (uint32_t)blocks) ++l.shift;
  l.magic = (uint32_t)((((uint64_t)1 << l.shift) + blocks - 1) / blocks);
  return l;
}

}  // namespace moe
