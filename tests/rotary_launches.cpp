// Prints the launches of the rotary kernels: one line "T heads kv_heads head_dim pairs interleaved" in, one line out.
#include <cstdio>

#include "../nvfp4_weight_quantized_amd/csrc/rotary_launch.h"

int main() {
  long long T, heads, hkv, D, pairs, inter;
  while (std::scanf("%lld %lld %lld %lld %lld %lld", &T, &heads, &hkv, &D, &pairs, &inter) == 6) {
    const moe::RotaryLaunch r = moe::plan_rotary(T, heads, D, pairs, inter);
    const moe::AppendRotaryLaunch a = moe::plan_append_rotary(T, heads, hkv, D, pairs, inter);
    std::printf("{\"pieces\": %d, \"per_block\": %d, \"blocks\": %lld, \"fits\": %d, \"quads\": %d, \"k_per\": %d, "
                "\"k_tokens\": %d, \"q\": %lld, \"k\": %lld, \"v\": %lld, \"append_blocks\": %lld, \"append_fits\": %d, "
                "\"threads\": %d, \"entries\": %d}\n",
                r.pieces, r.per_block, (long long)r.blocks, moe::rotary_fits(r.blocks), a.quads, a.k_per, a.k_tokens,
                (long long)a.q, (long long)a.k, (long long)a.v, (long long)a.blocks, moe::rotary_fits(a.blocks),
                moe::kRotaryThreads, moe::kRotaryEntries);
  }
}
