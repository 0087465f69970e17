// The launches of mm_id_sort, a rule on sizes alone (host code without HIP).
#pragma once

#include <stdint.h>

namespace mmk {

constexpr uint32_t kSortSlots = 8;  // slots of a token that the one launch counts in a round

// 1: sort_small alone. Each of its m blocks reads all m * top_k ids once a round,
// rounds one after the other, and a round of few ids still costs its memory
// round trip and two barriers, about 2.7 us. 2: the plan first. Measured in a
// graph, rows of 512 bf16, 64 experts, one launch against two (us):
//   rounds: 1 x 8 slots 4.3 and 6.1, 1 x 16 6.9 and 7.3, 1 x 32 12.2 and 9.7,
//     1 x 64 22.9 and 14.8, 128 x 16 8.0 and 8.3, 128 x 32 16.6 and 11.4;
//   ids read: 512 x 8 7.7 and 8.0, 256 x 16 9.8 and 9.0, 362 x 16 14.6 and 9.2,
//     724 x 4 6.9 and 6.9, 1024 x 2 6.7 and 6.3.
// The pieces of a wide row repeat the count beside each other, below the time
// of the copy, and have no part in the rule (512 x 8 f32 rows of 8192, four
// pieces: 28.9 and 30.4; 1024 x 2 bf16 rows of 8192: 12.6 and 12.8).
constexpr uint32_t kSmallRounds = 2;
constexpr uint64_t kSmallReads = 1u << 21;
inline int sort_launches(uint32_t m, uint32_t top_k) {
    const uint64_t rounds = ((uint64_t)top_k + kSortSlots - 1) / kSortSlots;
    // m * top_k < 2^31, so the reads of at most two rounds fit 64 bits.
    return rounds <= kSmallRounds && (uint64_t)m * top_k * m * rounds <= kSmallReads ? 1 : 2;
}

}  // namespace mmk
