// Tiles of 32 tokens of one head: which of them make groups of four whose places in a
// page follow each other (kv.hip, kv4.hip).
#pragma once
#include "q8k_device.h"

namespace q8k {

constexpr int TILE = 32, FOURS = TILE / 4;
// Tokens of a tile (lane t: token t's slot, -1: none) that begin a group of
// four, and those in none.
struct Groups {
    uint64_t fours, singles;
};
__device__ __forceinline__ Groups groups_of(const int* slots, int lane) {
    const int s = lane < TILE ? slots[lane] : -1;
    bool four = s >= 0 && (s & 3) == 0 && lane + 3 < TILE;
    if (four) four = slots[lane + 1] == s + 1 && slots[lane + 2] == s + 2 && slots[lane + 3] == s + 3;
    Groups g;
    g.fours = __ballot(four);
    g.singles = __ballot(s >= 0) & ~(g.fours | g.fours << 1 | g.fours << 2 | g.fours << 3);
    return g;
}
// The token of the n-th group (n-th bit of the mask), -1 behind the last: lane
// t's entry is written by it.
__device__ __forceinline__ void list_groups(uint64_t fours, int lane, int* list) {
    if (lane < FOURS && lane >= __popcll(fours)) list[lane] = -1;
    if (fours >> lane & 1) list[__popcll(fours & ((1ull << lane) - 1))] = lane;
}
// Rows of four bytes as columns: w[e] byte i becomes word i byte e.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
    const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    w[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
    w[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
    w[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
    w[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

}  // namespace q8k
