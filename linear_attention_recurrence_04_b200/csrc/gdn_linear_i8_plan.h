// gdn_linear_i8_plan.h -- which kernel takes a product of 8-bit integers. Plain
// host code without CUDA, so that tests can ask it which shapes reach which form.
#pragma once

#include <cstdint>

namespace gdn {

constexpr int kI8TileChannels = 128;   // output channels of a split tile
constexpr int kI8MaxSplits = 8;        // CTAs of a cluster that share a split tile

// W warps share a row so that long rows are on their way at once: at one
// token 2048 x 4096 takes 2.4 with 4, 2.6 with 2 and 4.2 with one,
// 4096 x 2048 3.3, 2.4 and 3.5, 2048 x 512 1.7, 1.5 and 1.3. Where another
// number is better: 8 tokens of 4096 x 2048 take 4.5 with 2 and 3.8 with one.
inline int vec_warps(int64_t K) { return K >= 4096 ? 4 : K >= 1024 ? 2 : 1; }

// Which kernel takes a product.
struct PlanI8 {
    enum Form { kVec, kSplit, kPair } form;
    int tile;      // split: tokens a tile; pair: channels a tile
    int splits;    // split: CTAs of a cluster
};

// The form with the least device time by a model of it (microseconds, graph
// replays on a B200, fitted to 50 shapes between 1 x 64 x 2048 and
// 16384 x 8192 x 2048; sums are exact, so the choice never shows in a result).
//   vec    a wave of warps (16 an SM) takes 0.4 + 0.39 per 1000 bytes of its
//          rows, after 1.1: 256 x 64 x 2048 in 2.5 against 3.6 (split), but
//          64 x 1024 x 1024 in 3.6 against 3.3. Calls of at most 4 tokens
//          always: 1 x 8192 x 2048 in 3.7 against 5.5.
//   split  a wave of CTAs starts and ends in 1.75 .. 2.9 and spends 0.27 ..
//          0.5 on 256 bytes of K; adding over a cluster costs 1.6 .. 2.9 more:
//          16 x 256 x 8192 in 4.3 with 8 CTAs against 10 with one, but
//          64 x 4096 x 2048 in 6.0 with 4 against 5.0 with one.
//   pair   starts and ends once, 4.9 or 5.6, and overlaps its tiles:
//          1024 x 8192 x 2048 in 18.2 against 29.5 (split), but
//          256 x 4096 x 2048 in 7.7 against 5.8.
inline PlanI8 plan_i8(int64_t M, int64_t N, int64_t K, int64_t sms) {
    if (M <= 4) return {PlanI8::kVec, 0, 0};
    const auto waves = [](int64_t n, int64_t at_once) {
        return static_cast<float>((n + at_once - 1) / at_once);
    };
    const float steps = waves(K, 256);
    PlanI8 best = {PlanI8::kVec, 0, 0};
    const int w = vec_warps(K), r = w == 4 ? 4 : 2;
    float least = 1.1f + waves((M + 7) / 8 * ((N + r - 1) / r) * w, 16 * sms) *
                             (0.4f + 0.00039f * K * r / w);
    const auto consider = [&](float t, PlanI8 p) {
        if (t < least) { least = t; best = p; }
    };
    struct { int tokens; float ends, step; } const tiles[] = {
        {16, 1.75f, 0.275f}, {32, 1.9f, 0.29f}, {64, 2.25f, 0.42f}, {128, 2.9f, 0.5f}};
    for (const auto& t : tiles) {
        if (t.tokens > 16 && t.tokens >= 2 * M) break;
        const int64_t n = ((N + kI8TileChannels - 1) / kI8TileChannels) * ((M + t.tokens - 1) / t.tokens);
        consider(waves(n, sms) * (t.ends + steps * t.step), {PlanI8::kSplit, t.tokens, 1});
        // (clusters of 8 find room for 96 CTAs at once at most)
        for (int s = 2; s <= kI8MaxSplits; s *= 2) {
            if (s > steps || n * s > (s == 8 ? 96 : sms)) break;
            consider(t.ends + waves(static_cast<int64_t>(steps), s) * t.step + 1.4f +
                         0.012f * t.tokens,
                     {PlanI8::kSplit, t.tokens, s});
        }
    }
    if (M > 128) {
        const int64_t rows = (M + 255) / 256;
        const float w1 = waves(rows * ((N + 127) / 128), sms / 2);
        const float w2 = waves(rows * ((N + 255) / 256), sms / 2);
        consider(4.1f + w1 * (0.8f + 0.39f * steps), {PlanI8::kPair, 128, 1});
        consider(5.1f + w2 * (0.5f + 0.72f * steps), {PlanI8::kPair, 256, 1});
    }
    return best;
}

}  // namespace gdn
