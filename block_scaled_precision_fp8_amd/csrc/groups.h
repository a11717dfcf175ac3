// groups.h -- groups of rows given by their offsets on the device, as the grouped
// kernels read them.
//
// Group e holds the rows offsets[e] .. offsets[e + 1] - 1.  The array is only known
// on the device, so whatever it holds must keep every access in bounds: starts are
// clamped to 0 .. limit and never go back, so that groups are disjoint and their
// sizes add up to at most limit.  In a transpose a group's rows become
// columns from a multiple of 128 on (`block` counts 128s) and its scale bytes whole
// words of four blocks (`word`).
#pragma once

#include "internal.h"

namespace bsfp8 {
namespace groups {

constexpr int kMaxGroups = 1024;

// One group, in a lane of its own.
struct Lane {
    int e, start, rows;
    int tile, tiles;             // the first of its tiles of 2^SHIFT rows, and how many
    int word;                    // the first of its words of four tiles
};

// Inclusive scans over a wave, of values >= 0: within 16 lanes, then across them, by lane moves on the
// VALU (through LDS shuffles three scans take about a microsecond, which every workgroup waits for).
template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
template <class F>
__device__ __forceinline__ int scan(int v, F&& f) {
    v = f(v, moved<0x111, 0xF>(v));              // row_shr 1, 2, 4, 8
    v = f(v, moved<0x112, 0xF>(v));
    v = f(v, moved<0x114, 0xF>(v));
    v = f(v, moved<0x118, 0xF>(v));
    v = f(v, moved<0x142, 0xA>(v));              // lane 15 of a row to the next one
    return f(v, moved<0x143, 0xC>(v));           // lane 31 to the upper half
}
__device__ __forceinline__ int scan_add(int v) {
    return scan(v, [](int a, int b) { return a + b; });
}
__device__ __forceinline__ int scan_max(int v) {
    return scan(v, [](int a, int b) { return max(a, b); });
}

// Calls f(Lane, in) for 64 groups at a time, in order, by a whole wave, until it
// returns true; in: the lane holds a group.  T: a tile is T rows.
template <int T, class F>
__device__ __forceinline__ void for_each(const int32_t* __restrict__ offsets, int count, int limit, F&& f) {
    const int lane = threadIdx.x & 63;
    int start = min(max(offsets[0], 0), limit), tile = 0, word = 0;
    for (int e0 = 0; e0 < count; e0 += 64) {
        const int e = e0 + lane;
        const bool in = e < count;
        const int end = scan_max(max(min(in ? offsets[e + 1] : 0, limit), start));
        const int before = __shfl_up(end, 1);
        Lane g;
        g.e = e;
        g.start = lane == 0 ? start : before;
        g.rows = end - g.start;
        g.tiles = (g.rows + T - 1) / T;
        const int words = (g.tiles + 3) >> 2;
        const int t = scan_add(g.tiles), w = scan_add(words);
        g.tile = tile + t - g.tiles;
        g.word = word + w - words;
        if (f(g, in)) return;
        start = __builtin_amdgcn_readlane(end, 63);
        tile += __builtin_amdgcn_readlane(t, 63);
        word += __builtin_amdgcn_readlane(w, 63);
    }
}

// The lane's group in every lane's (scalar) registers.
__device__ __forceinline__ Lane broadcast(const Lane& g, int lane) {
    Lane o;
    o.e = __builtin_amdgcn_readlane(g.e, lane);
    o.start = __builtin_amdgcn_readlane(g.start, lane);
    o.rows = __builtin_amdgcn_readlane(g.rows, lane);
    o.tile = __builtin_amdgcn_readlane(g.tile, lane);
    o.tiles = __builtin_amdgcn_readlane(g.tiles, lane);
    o.word = __builtin_amdgcn_readlane(g.word, lane);
    return o;
}

// The group that tile t belongs to; rows = 0 where there are fewer tiles.
template <int T>
__device__ __forceinline__ Lane of_tile(const int32_t* offsets, int count, int limit, int t) {
    Lane found{};
    for_each<T>(offsets, count, limit, [&](const Lane& g, bool in) {
        const uint64_t hit = __ballot(in && t < g.tile + g.tiles);
        if (hit) found = broadcast(g, __builtin_ctzll(hit));
        return hit != 0;
    });
    return found;
}
// Group e < count.
template <int T>
__device__ __forceinline__ Lane at(const int32_t* offsets, int count, int limit, int e) {
    Lane found{};
    for_each<T>(offsets, count, limit, [&](const Lane& g, bool) {
        if (e >= g.e - static_cast<int>(threadIdx.x & 63) + 64) return false;
        found = broadcast(g, e & 63);
        return true;
    });
    return found;
}

}  // namespace groups
}  // namespace bsfp8
