// Sizes of the paged key/value cache that host and device code share.
#pragma once

namespace moe {

constexpr int kKvMaxRequests = 4096;
constexpr int kKvUnit = 32;   // positions per unit of a page (36 * head_dim bytes)

}  // namespace moe
