// adapter.cuh -- arguments and device helpers shared by the low-rank adapter kernels.
#pragma once

#include "nq_common.cuh"

namespace nq {

// One product pair of the adapters, forward or its transpose:
//   t[m] = scale_a P_a z[m],  out[m] = base[m] + Q_a t[m],  a = the adapter of row m
// forward: z = x, P = A, Q = B; backward: z = ybar, P = B^T, Q = A^T, t = u.
struct AdapterArgs {
    const int32_t* rows;     // [M] rows grouped by adapter, rows without one last
    const int32_t* offsets;  // [n + 1] where each adapter's rows begin in `rows`
    const uint16_t* z;       // [M][K] bf16
    const uint16_t* base;    // [M][N] bf16
    uint16_t* out;           // [M][N] bf16, may be base; nullptr: only t is wanted
    float* t;                // [M][rank] fp32 or nullptr
    const uint16_t* A;       // [n][rank][lda] bf16
    const uint16_t* B;       // [n][d_out][ldb] bf16
    const float* scale;      // [n] or nullptr (ones)
    int64_t lda, ldb, d_in, d_out;
    int64_t K, N;            // widths of z and of base
    int64_t M;
    int n, rank;
    unsigned int* err;
    // For the sums over tokens on the tensor cores: u, and t_in [M][rank] fp32, as the sum of two bf16
    // values (split_for_sums), rows in the order of `rows` with every adapter's padded to a multiple of 16 by zeros:
    // part p of padded row i at parts + (p part_rows + i) part_ld.  nullptr: not wanted.
    const float* t_in;
    uint16_t* u_parts;
    uint16_t* t_parts;
    int64_t part_rows;
    int part_ld;  // 64 or 128
};

// Rows, list entries and padded rows are 32-bit numbers on the device: a group rounded up to a tile of
// 128, a step of up to 128 past its end, and a row of the second of two arrays of padded rows (a TMA
// coordinate) all fit.
static_assert(int64_t{NQ_ADAPTER_MAX_M} + 256 < INT32_MAX &&
                  2 * (int64_t{NQ_ADAPTER_MAX_M} + 15 * int64_t{NQ_ADAPTER_MAX_N}) < INT32_MAX,
              "row numbers in 32 bits");

// Padded rows of M rows in n groups, at most.
inline int64_t max_padded_rows(int64_t M, int64_t n) { return M + 15 * (n < M ? n : M); }

// Sum over the tokens of each adapter (a = blockIdx.y):
//   gA_a[r][j] = sum_m u[m][r] x[m][j],   gB_a[i][r] = sum_m ybar[m][i] t[m][r]
struct AdapterGradArgs {
    const int32_t* rows;
    const int32_t* offsets;
    const uint16_t* x;     // [M][d_in]
    const uint16_t* ybar;  // [M][d_out]
    const float* t;        // [M][rank]
    const float* u;        // [M][rank]
    uint16_t* gA;          // [n][rank][d_in] bf16 or nullptr
    uint16_t* gB;          // [n][d_out][rank] bf16 or nullptr
    int64_t d_in, d_out, M;
    int n, rank;
    unsigned int* err;
};

// A run of at most `rows_per_tile` entries of `rows` that share an adapter.
struct AdapterTile {
    int adapter;  // n: rows without an adapter; -1: no such tile
    int first;    // index into rows
    int count;
    int padded;   // padded row of the tile's first (of every group's rows in multiples of 16)
};

// Bounds of adapter a's entries in `rows`, forced into 0 <= first <= last <= M whatever the
// offsets say; a == n: the rows after the last adapter's.  Offsets outside that order are
// reported, and false is returned.  Groups whose predecessors are all in order hold M rows at most between
// them; one pair alone says nothing about that (0, M, 0, M), so the scans below count every
// group from the first bad pair on as empty.
__device__ __forceinline__ bool adapter_bounds(const int32_t* offsets, int n, int64_t M, int a, int& first, int& last,
                                               unsigned int* err) {
    const int64_t lo = offsets[a], hi = a < n ? static_cast<int64_t>(offsets[a + 1]) : M;
    const bool ok = lo >= 0 && lo <= hi && hi <= M && (a > 0 || lo == 0);
    if (!ok) flag_error(err, kErrIndex);
    first = static_cast<int>(ok ? lo : 0);
    last = static_cast<int>(ok ? hi : 0);
    return ok;
}

// Tile number `tile` when every adapter's rows are cut into tiles of rows_per_tile and those
// without one into tiles of none_per_tile, groups in order.  A whole warp calls it; 32 L groups are
// scanned at a time, L neighbours a lane.
template <int L>
__device__ __forceinline__ AdapterTile find_tile_by(const int32_t* offsets, int n, int64_t M, int rows_per_tile,
                                                    int none_per_tile, int tile, unsigned int* err) {
    const int lane = threadIdx.x & 31;
    int before = 0;  // tiles of the groups before this batch
    int padded = 0;  // and their rows in multiples of 16
    for (int a0 = 0; a0 <= n; a0 += 32 * L) {
        int first[L], last[L], tiles[L], mine = 0, rows16 = 0;
        bool ok = true;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int a = a0 + L * lane + i;
            first[i] = last[i] = 0;
            if (a <= n) ok = adapter_bounds(offsets, n, M, a, first[i], last[i], err) && ok;
            if (!ok) first[i] = last[i] = 0;
        }
        const unsigned bad = __ballot_sync(0xFFFFFFFFu, !ok);
        if (bad != 0u && lane >= __ffs(bad)) {  // lanes after the first with a bad pair
#pragma unroll
            for (int i = 0; i < L; ++i) first[i] = last[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int per = a0 + L * lane + i < n ? rows_per_tile : none_per_tile;
            tiles[i] = (last[i] - first[i] + per - 1) / per;
            mine += tiles[i];
            rows16 += (last[i] - first[i] + 15) & ~15;
        }
        int upto = mine;  // inclusive sum over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
        const int local = tile - before;
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, local < upto);
        if (hit) {
            const int src = __ffs(hit) - 1;
            AdapterTile t;
            t.padded = padded + static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, lane < src ? rows16 : 0));
            // the lane that has it looks through its groups
            int rest = local - (upto - mine);
            t.adapter = -1;
            t.first = t.count = 0;
            int in_lane = 0;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (t.adapter < 0 && rest < tiles[i]) {
                    const int per = a0 + L * lane + i < n ? rows_per_tile : none_per_tile;
                    t.adapter = a0 + L * lane + i;
                    t.first = first[i] + rest * per;
                    t.count = min(per, last[i] - t.first);
                    in_lane += rest * per;
                } else if (t.adapter < 0) {
                    rest -= tiles[i];
                    in_lane += (last[i] - first[i] + 15) & ~15;
                }
            }
            t.adapter = __shfl_sync(0xFFFFFFFFu, t.adapter, src);
            t.first = __shfl_sync(0xFFFFFFFFu, t.first, src);
            t.count = __shfl_sync(0xFFFFFFFFu, t.count, src);
            t.padded += __shfl_sync(0xFFFFFFFFu, in_lane, src);
            return t;
        }
        if (bad != 0u) break;
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
        padded += static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, rows16));
    }
    return {-1, 0, 0, 0};
}

// One group a lane where that is all of them (the common case, with the least latency).
__device__ __forceinline__ AdapterTile find_tile(const int32_t* offsets, int n, int64_t M, int rows_per_tile,
                                                 int none_per_tile, int tile, unsigned int* err) {
    return n < 32 ? find_tile_by<1>(offsets, n, M, rows_per_tile, none_per_tile, tile, err)
                  : find_tile_by<4>(offsets, n, M, rows_per_tile, none_per_tile, tile, err);
}

// Adapter a's bounds in `rows` and its first padded row; no rows after a bad pair.  A whole warp calls it.
__device__ __forceinline__ int find_group(const int32_t* offsets, int n, int64_t M, int adapter, int& first, int& last,
                                          unsigned int* err) {
    const int lane = threadIdx.x & 31;
    int padded = 0;
    for (int a0 = 0; a0 < adapter; a0 += 32) {
        int f = 0, l = 0;
        const bool ok = a0 + lane >= adapter || adapter_bounds(offsets, n, M, a0 + lane, f, l, err);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
            first = last = 0;
            return 0;
        }
        padded += static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, (l - f + 15) & ~15));
    }
    adapter_bounds(offsets, n, M, adapter, first, last, err);
    return padded;
}

// Tiles of M rows in n adapters and "none": with one tile size an upper bound for any grouping, which a grid
// without a loop needs.  Where none_per_tile is the smaller, the larger of the two extremes (every row
// listed, none listed): a mixture can make more, and the clusters loop over them.
inline int64_t max_adapter_tiles(int64_t M, int64_t n, int rows_per_tile, int none_per_tile) {
    const int64_t groups = n + 1 < M ? n + 1 : M;
    const int64_t listed = (M - groups) / rows_per_tile + groups, none = (M - 1) / none_per_tile + 1;
    return listed > none ? listed : none;
}

// Entry i of `rows`, or -1 (reported) when it is not a row.
__device__ __forceinline__ int checked_row(const int32_t* rows, int64_t i, int64_t M, unsigned int* err) {
    const int r = rows[i];
    if (r >= 0 && r < M) return r;
    flag_error(err, kErrIndex);
    return -1;
}

// ------------------------------------------------------------------ fp32 values in two bf16 parts
// What v's bf16 part leaves of it (nothing of an infinity).
__device__ __forceinline__ float rest_of(float v, uint32_t part) {
    const float p = __uint_as_float(part);
    return isinf(p) ? 0.f : v - p;
}

// Two fp32 values as the sum of two bf16 values each, for products that keep the parts apart (join_parts).
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(rest_of(a, hi << 16), rest_of(b, hi & 0xFFFF0000u));
}

// A sum over first parts and the same over second parts, which have accumulators of their own.  Against an
// infinity the second parts, which may be 0 or of the other sign, add up to an infinity or NaN that
// the value itself does not have; the first parts alone then give its infinity or NaN.
__device__ __forceinline__ float join_parts(uint32_t hi, uint32_t lo) {
    const float l = __uint_as_float(lo);
    return __uint_as_float(hi) + (isfinite(l) ? l : 0.f);
}

// The same for products that share an accumulator: the second part has the value's sign and is 0 only of a
// 0, so that against an infinity the parts agree.  The first is cut instead of rounded, which costs one bit
// of 17, and the smallest number, 2^-133, stands in for a second part of nothing: off by 2^-16 of the
// value or 2^-133 at most.
__device__ __forceinline__ uint32_t second_part(float v) {
    const uint32_t bits = __float_as_uint(v);
    const float first = __uint_as_float(bits & 0xFFFF0000u);
    const uint32_t rest = float_to_bf16_bits(v == first ? 0.f : v - first);
    return (rest & 0x7FFFu) != 0u || v == 0.f ? rest : (bits >> 16 & 0x8000u) | 1u;
}
__device__ __forceinline__ void split_bf16_same_sign(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    lo = second_part(a) | second_part(b) << 16;
}

// The sums over tokens have room in TMEM for two units of work and for accumulators of both parts up to
// rank 64; above it the parts share them.
__device__ __forceinline__ bool sums_keep_parts_apart(int part_ld) { return part_ld == 64; }
__device__ __forceinline__ void split_for_sums(int part_ld, float a, float b, uint32_t& hi, uint32_t& lo) {
    if (sums_keep_parts_apart(part_ld))
        split_bf16(a, b, hi, lo);
    else
        split_bf16_same_sign(a, b, hi, lo);
}

}  // namespace nq
