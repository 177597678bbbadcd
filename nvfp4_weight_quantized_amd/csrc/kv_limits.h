// Sizes of the paged key/value cache that host and device code share.
#pragma once

namespace moe {

constexpr int kKvMaxRequests = 4096;
constexpr int kKvMaxSelectPages = 16384;   // pages of a row of the block table that a choice looks at
constexpr int kKvMaxSelected = 1024;       // pages chosen for a row
constexpr long long kKvAppendQuadThreads = 1 << 19;   // rows * groups of an append from which quads are taken (kv_cache.hip)
constexpr int kKvUnit = 32;   // positions per unit of a page (36 * head_dim bytes)

}  // namespace moe
