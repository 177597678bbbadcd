// Prints the launches of attention calls: one line "T R G hkv D table_units" in, per launch one line out.
#include <cstdio>

#include "../nvfp4_weight_quantized_amd/csrc/kv_launch.h"

int main() {
  long long T, R, G, hkv, D, units;
  while (std::scanf("%lld %lld %lld %lld %lld %lld", &T, &R, &G, &hkv, &D, &units) == 6) {
    const moe::Launches x = moe::plan_launches(T, R, G, hkv, D, units);
    for (int i = 0; i < x.n; ++i) {
      const moe::Launch& p = x.l[i];
      std::printf("{\"shares\": %d, \"whole\": %d, \"rs\": %d, \"bm\": %d, \"target\": %d, \"min_rows\": %d, \"max_rows\": %d, "
                  "\"grid\": %lld, \"tiles\": %lld, \"join\": %lld, \"bytes\": %zu}%s",
                  p.shares, p.whole, p.rs, p.s.bm, p.s.target, p.s.min_rows, p.s.max_rows, (long long)p.grid,
                  (long long)p.tiles, (long long)p.join, p.bytes, i + 1 < x.n ? ", " : "");
    }
    std::printf("\n");
  }
}
