// mx_block_group.h -- groups of rows given by their ends in device memory: which
// group a workgroup's tile belongs to.
//
// Group i is the rows from the largest end before it (0 for the first) to its own
// end, ends taken as at most `rows` and at least the ends before them; so whatever
// the memory holds, no group reaches past the rows and none overlaps another.  A
// wave takes 256 ends at a time, four in a row per lane, so that up to 256 groups
// cost one read's latency, and scans them by DPP: a running maximum, and a running
// sum of the groups' sizes in units of UNIT rows, rounded up.
#pragma once
#include "mx_block_internal.h"

namespace mx {
namespace {

template <int CTRL, int ROWS>
__device__ __forceinline__ int scan_move(int v) {  // 0 for lanes without a source
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
// inclusive scans over the wave: shifts by 1, 2, 4, 8 within rows of 16 lanes, then the rows before
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
    v = op(v, scan_move<0x111, 0xF>(v));
    v = op(v, scan_move<0x112, 0xF>(v));
    v = op(v, scan_move<0x114, 0xF>(v));
    v = op(v, scan_move<0x118, 0xF>(v));
    v = op(v, scan_move<0x142, 0xA>(v));  // last lane of a row to the next row: rows 1 and 3
    v = op(v, scan_move<0x143, 0xC>(v));  // lane 31 to rows 2 and 3
    return v;
}

struct Group {
    int index, start, count;  // rows start .. start + count - 1
    int first;                // units of the groups before it
};

// v[j] of a lane, j and the lane scalar
__device__ __forceinline__ int pick(const int (&v)[4], int lane, int j) {
    const int a = __builtin_amdgcn_readlane(v[0], lane), b = __builtin_amdgcn_readlane(v[1], lane);
    const int c = __builtin_amdgcn_readlane(v[2], lane), d = __builtin_amdgcn_readlane(v[3], lane);
    return j == 0 ? a : j == 1 ? b : j == 2 ? c : d;
}

// 256 groups from g0 on, four per lane
template <int UNIT>
struct GroupChunk {
    int end[4], incl[4];     // ends of the groups; units up to and with each
    int start, before;       // the lane's first group: its first row, the units before it
    int carry_row = 0, carry_units = 0;  // scalar: the last end and all units up to here

    __device__ __forceinline__ void load(const int32_t *ends, int groups, int rows, int g0) {
        const int lane = threadIdx.x & 63, i = g0 + 4 * lane;
        if (i + 4 <= groups) {
            __builtin_memcpy(end, ends + i, 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++) end[j] = i + j < groups ? ends[i + j] : 0;
        }
        int m = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) end[j] = m = max(m, min(end[j], rows));
        m = wave_scan(m, [](int a, int b) { return max(a, b); });
        start = __shfl_up(m, 1);
        start = max(lane ? start : 0, carry_row);
        int at = start, units = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            end[j] = max(end[j], start);
            incl[j] = units += (int)(((uint32_t)(end[j] - at) + UNIT - 1) / UNIT);
            at = end[j];
        }
        const int sum = wave_scan(units, [](int a, int b) { return a + b; });
        before = sum - units + carry_units;
#pragma unroll
        for (int j = 0; j < 4; j++) incl[j] += before;
        carry_row = __builtin_amdgcn_readlane(at, 63);
        carry_units += __builtin_amdgcn_readlane(sum, 63);
    }
    // group number 4 lane + j of these
    __device__ __forceinline__ Group at(int g0, int lane, int j) const {
        const int e = pick(end, lane, j);
        const int s = j ? pick(end, lane, j - 1) : __builtin_amdgcn_readlane(start, lane);
        const int f = j ? pick(incl, lane, j - 1) : __builtin_amdgcn_readlane(before, lane);
        return {g0 + 4 * lane + j, s, e - s, f};
    }
};

// units of all groups; `c` is left holding the first 256 groups
template <int UNIT>
__device__ __forceinline__ int group_units(GroupChunk<UNIT> &c, const int32_t *ends, int groups, int rows) {
    c.load(ends, groups, rows, 0);
    if (groups <= 256) return c.carry_units;
    GroupChunk<UNIT> d = c;
    for (int g0 = 256; g0 < groups; g0 += 256) d.load(ends, groups, rows, g0);
    return d.carry_units;
}
// the group that unit `want` (of the units counted) belongs to
template <int UNIT>
__device__ __forceinline__ Group group_of_unit(GroupChunk<UNIT> c, const int32_t *ends, int groups, int rows, int want) {
    for (int g0 = 0;; g0 += 256) {
        const uint64_t m = __ballot(c.incl[3] > want);
        if (m) {
            const int lane = __builtin_ctzll(m);
            const int j = (__builtin_amdgcn_readlane(c.incl[0], lane) <= want) + (__builtin_amdgcn_readlane(c.incl[1], lane) <= want) +
                          (__builtin_amdgcn_readlane(c.incl[2], lane) <= want);
            return c.at(g0, lane, j);
        }
        if (g0 + 256 >= groups) return {0, 0, 0, 0};  // not reached: want is below the sum
        c.load(ends, groups, rows, g0 + 256);
    }
}
// group `index`
template <int UNIT>
__device__ __forceinline__ Group group_number(const int32_t *ends, int groups, int rows, int index) {
    GroupChunk<UNIT> c;
    c.load(ends, groups, rows, 0);
    int g0 = 0;
    for (; g0 + 256 <= index; g0 += 256) c.load(ends, groups, rows, g0 + 256);
    return c.at(g0, (index - g0) >> 2, (index - g0) & 3);
}

}  // namespace
}  // namespace mx
