// mx_block_group.h -- groups of rows given by their ends in device memory: which
// group a workgroup's tile belongs to.
//
// Group i is the rows from the largest end before it (0 for the first) to its own
// end, ends taken as at most `rows` and at least the ends before them; so whatever
// the memory holds, no group reaches past the rows and none overlaps another.  A
// wave reads 64 ends at a time and scans them by DPP: a running maximum, and a
// running sum of the groups' sizes in units of UNIT rows, rounded up.
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

// 64 groups, one per lane; all values of a lane but the carries, which are scalar
template <int UNIT>
struct GroupChunk {
    int start, count, units, incl;
    int carry_row = 0, carry_units = 0;

    __device__ __forceinline__ void load(const int32_t *ends, int groups, int rows, int g0) {
        const int i = g0 + (int)(threadIdx.x & 63);
        const int e = i < groups ? min(max(ends[i], 0), rows) : 0;
        const int m = max(wave_scan(e, [](int a, int b) { return max(a, b); }), carry_row);
        start = __shfl_up(m, 1);
        if ((threadIdx.x & 63) == 0) start = carry_row;
        count = m - start;
        units = (int)(((uint32_t)count + UNIT - 1) / UNIT);
        incl = wave_scan(units, [](int a, int b) { return a + b; }) + carry_units;
        carry_row = __builtin_amdgcn_readlane(m, 63);
        carry_units = __builtin_amdgcn_readlane(incl, 63);
    }
    __device__ __forceinline__ Group at(int g0, int lane) const {
        return {g0 + lane, __builtin_amdgcn_readlane(start, lane), __builtin_amdgcn_readlane(count, lane),
                __builtin_amdgcn_readlane(incl, lane) - __builtin_amdgcn_readlane(units, lane)};
    }
};

// units of all groups; `c` is left holding the first 64 groups
template <int UNIT>
__device__ __forceinline__ int group_units(GroupChunk<UNIT> &c, const int32_t *ends, int groups, int rows) {
    c.load(ends, groups, rows, 0);
    GroupChunk<UNIT> d = c;
    for (int g0 = 64; g0 < groups; g0 += 64) d.load(ends, groups, rows, g0);
    return d.carry_units;
}
// the group that unit `want` (of the units counted) belongs to
template <int UNIT>
__device__ __forceinline__ Group group_of_unit(GroupChunk<UNIT> c, const int32_t *ends, int groups, int rows, int want) {
    for (int g0 = 0;; g0 += 64) {
        const uint64_t m = __ballot(c.incl > want);
        if (m) return c.at(g0, __builtin_ctzll(m));
        if (g0 + 64 >= groups) return {0, 0, 0, 0};  // not reached: want is below the sum
        c.load(ends, groups, rows, g0 + 64);
    }
}
// group `index`
template <int UNIT>
__device__ __forceinline__ Group group_number(const int32_t *ends, int groups, int rows, int index) {
    GroupChunk<UNIT> c;
    c.load(ends, groups, rows, 0);
    int g0 = 0;
    for (; g0 + 64 <= index; g0 += 64) c.load(ends, groups, rows, g0 + 64);
    return c.at(g0, index - g0);
}

}  // namespace
}  // namespace mx
