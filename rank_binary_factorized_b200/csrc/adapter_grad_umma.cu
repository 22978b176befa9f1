// adapter_grad_umma.cu -- the adapters' own gradients on the tensor cores (tcgen05):
//
//   gA_a[r][j] = sum_m u[m][r] x[m][j],   gB_a[i][r] = sum_m ybar[m][i] t[m][r]   (a's rows m)
//
// Both are z^T t with the tokens as the MMA's K: D[256 columns of z][rank], z = x with u or ybar with
// t.  z is read once from HBM (2 bytes an element against 2 rank flops) and bounds the kernel; u and
// t, two bf16 parts each (16 bits: the products keep more than the bf16 result does), come from L2
// for every block of 256 columns, which is why a block is that wide and not 128.
//
// A work unit is one adapter and 256 columns of x or ybar; the blocks take units in turn.  Warp 0
// loads 64 tokens at a time (z: TMA boxes where rows follow one another, row gathers where not; rows
// past the group's last arrive as zeros, so that nothing of another row can reach the sum), warp 1
// issues the MMAs, warps 2..5 round the accumulators to bf16 and store them.  TMEM holds two units, so
// that one is stored while the next is summed; up to rank 64 the two parts of u and t have
// accumulators of their own, which are cut half as often (at rank 128 that would leave room for one
// unit: the backward pass of 2500 rows of a 7B gate in three even groups took 92 us so, 84 as it is).
// Where the units are fewer than the multiprocessors, several blocks share the tokens of one and a
// small kernel adds their sums.
// Measured (B200): 4096 rows of a 70B gate at rank 64 63 us, 302 MB of x and ybar at 4.8 TB/s, 0.73 of the
// measured copy rate (and as much again of u and t from L2).
#include <algorithm>
#include <atomic>

#include "adapter_tc.cuh"

namespace nq {

constexpr int kWgCols = 256;                // columns of z of a unit: two MMA tiles
constexpr int kWgTok = 64;                  // tokens of a slot
constexpr uint32_t kWgPanel = kWgTok * 128; // 64 tokens x 64 bf16
constexpr int kWgThreads = 192;
constexpr uint32_t kWgUnitCols = 256;       // TMEM columns of a unit
constexpr int kWgMaxSlots = 4;
constexpr int kWgGroups = 1024;             // groups whose bounds are kept in shared memory

struct AdapterWgradArgs {
    AdapterGradArgs g;
    int64_t part_rows;
    int in_tiles, out_tiles;  // units of d_in (0 without gA) and of d_out (0 without gB)
    int slots;
    uint32_t slot_bytes;
    int panels, r16;
    uint32_t acc_cols;        // TMEM columns of a unit's two accumulators (of one part of u or t, if apart)
    int splits;               // blocks that share the tokens of a unit
    float* partial;           // splits > 1: [splits] sums of gA [n][rank][d_in], then of gB [n][d_out][rank]
    int64_t split_stride, gb_at;
};

__global__ void __launch_bounds__(kWgThreads, 1)
    adapter_wgrad_umma_kernel(const __grid_constant__ CUtensorMap x64, const __grid_constant__ CUtensorMap x32,
                              const __grid_constant__ CUtensorMap x1, const __grid_constant__ CUtensorMap y64,
                              const __grid_constant__ CUtensorMap y32, const __grid_constant__ CUtensorMap y1,
                              const __grid_constant__ CUtensorMap map_u, const __grid_constant__ CUtensorMap map_t,
                              const AdapterWgradArgs wa) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const AdapterGradArgs& g = wa.g;
    const uint32_t smem_base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    const int slots = wa.slots, panels = wa.panels, r16 = wa.r16;
    const uint32_t bars = smem_base + slots * wa.slot_bytes;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (kWgMaxSlots + s); };
    auto acc_full = [&](int i) { return bars + 8u * (2 * kWgMaxSlots + i); };
    auto acc_empty = [&](int i) { return bars + 8u * (2 * kWgMaxSlots + 2 + i); };
    const uint32_t drain = bars + 8u * (2 * kWgMaxSlots + 4), tmem_slot = drain + 8u;
    // bounds of every adapter's rows (where there are not too many): first, last, first padded row
    int(*const bounds)[3] = reinterpret_cast<int(*)[3]>(smem_raw + (bars + 384u - tc::smem_u32(smem_raw)));
    const bool kept = g.n <= kWgGroups, sorted = g.n <= 64;
    int* const order = reinterpret_cast<int*>(smem_raw + (bars + 128u - tc::smem_u32(smem_raw)));  // of 64 at most
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned int* err = g.err;

    if (warp == 0) {
        if (lane < slots) {
            tc::mbar_init(full(lane), 1);
            tc::mbar_init(empty(lane), 1);
        } else if (lane == 8 || lane == 9) {
            tc::mbar_init(acc_full(lane - 8), 1);
            tc::mbar_init(acc_empty(lane - 8), 4);
        } else if (lane == 10) {
            tc::mbar_init(drain, 1);
        }
        tc::mbar_fence_init();
        __syncwarp();
    } else if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem_raw + (tmem_slot - tc::smem_u32(smem_raw)));
    const bool apart = sums_keep_parts_apart(panels * 64);
    const uint32_t second = apart ? wa.acc_cols : 0u;  // where the second parts' accumulators are
    const int per_adapter = wa.in_tiles + wa.out_tiles;
    const int64_t units = static_cast<int64_t>(per_adapter) * g.n * wa.splits;
    // tokens of split sp of a group, in slots
    auto share = [&](int rows, int sp, int& b0, int& b1) {
        const int64_t all = (rows + kWgTok - 1) / kWgTok;
        b0 = static_cast<int>(all * sp / wa.splits);
        b1 = static_cast<int>(all * (sp + 1) / wa.splits);
    };
    // The lists were written before the launch ahead of this one, which waited for its own predecessors
    // before it let this one start: they may be read before that launch is over.
    if (kept) {
        if (warp == 0) {
            int padded = 0;
            bool in_order = true;  // every pair before these 32
            for (int a0 = 0; a0 < g.n; a0 += 32) {
                int first = 0, last = 0;
                const bool pair = a0 + lane >= g.n || adapter_bounds(g.offsets, g.n, g.M, a0 + lane, first, last, err);
                const unsigned bad = __ballot_sync(0xFFFFFFFFu, !pair);
                if (!in_order || (bad != 0u && lane >= __ffs(bad) - 1)) first = last = 0;
                in_order = in_order && bad == 0u;
                const int rows16 = (last - first + 15) & ~15;
                int upto = rows16;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                    if (lane >= o) upto += v;
                }
                if (a0 + lane < g.n) {
                    bounds[a0 + lane][0] = first;
                    bounds[a0 + lane][1] = last;
                    bounds[a0 + lane][2] = padded + upto - rows16;
                }
                padded += __shfl_sync(0xFFFFFFFFu, upto, 31);
            }
            __syncwarp();
            // adapters by their number of rows, most first (equal ones by index)
            for (int i = lane; i < g.n && sorted; i += 32) {
                const int mine = bounds[i][1] - bounds[i][0];
                int place = 0;
                for (int j = 0; j < g.n; ++j) {
                    const int other = bounds[j][1] - bounds[j][0];
                    place += other > mine || (other == mine && j < i);
                }
                order[place] = i;
            }
        }
        __syncthreads();
    }
    pdl_wait();
    pdl_launch_dependents();
    // The blocks take units in turn, there and back, from the longest adapter's on: a block's last unit is
    // short where its others were long.
    auto unit_of = [&](int64_t round) {
        return round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    };
    auto adapter_of = [&](int64_t unit) {
        const int a = static_cast<int>(unit / wa.splits / per_adapter);
        return sorted ? order[a] : a;
    };
    auto group = [&](int adapter, int& first, int& last) {  // returns the first padded row (warp-wide)
        if (!kept) return find_group(g.offsets, g.n, g.M, adapter, first, last, err);
        first = bounds[adapter][0];
        last = bounds[adapter][1];
        return bounds[adapter][2];
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        uint32_t it = 0;
        int s = 0;
        bool ok = true;
        for (int64_t round = 0, unit; (unit = unit_of(round)) < units && ok; ++round) {
            const int sp = static_cast<int>(unit % wa.splits);
            const int adapter = adapter_of(unit);
            const int tile = static_cast<int>(unit / wa.splits % per_adapter);
            const bool is_a = tile < wa.in_tiles;
            const int col0 = (is_a ? tile : tile - wa.in_tiles) * kWgCols;
            const int width = static_cast<int>(is_a ? g.d_in : g.d_out);
            const int z_panels = min(kWgCols / 64, (width - col0 + 63) / 64);
            int first, last;
            const int padded = group(adapter, first, last);
            int b0, b1;
            share(last - first, sp, b0, b1);
            int32_t next[4];  // the next slot's entries, loaded a slot ahead
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = first + b0 * kWgTok + (lane & 15) * 4 + i;
                next[i] = e < last ? g.rows[e] : -1;
            }
            for (int e0 = first + b0 * kWgTok; e0 < min(last, first + b1 * kWgTok) && ok; e0 += kWgTok) {
                const int count = min(kWgTok, last - e0);
                // lane l < 16 holds entries 4 l .. 4 l + 3; rows past the last are given as M: zeros
                int32_t row[4];
                const int first32 = __shfl_sync(0xFFFFFFFFu, next[0], lane & 8);
                bool follow = true;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = (lane & 15) * 4 + i;
                    const bool ok_row = e < count && next[i] >= 0 && next[i] < g.M;
                    if (e < count && !ok_row) flag_error(err, kErrIndex);
                    follow = follow && ok_row && next[i] == first32 + (e & 31);
                    row[i] = ok_row ? next[i] : static_cast<int32_t>(g.M);
                    next[i] = e0 + kWgTok + e < last ? g.rows[e0 + kWgTok + e] : -1;
                }
                const uint32_t follows = __ballot_sync(0xFFFFFFFFu, follow || lane >= 16);
                const bool box = ((follows >> (lane & 8)) & 0xFFu) == 0xFFu;  // 32 rows one after the other
                const int32_t row0 = __shfl_sync(0xFFFFFFFFu, row[0], 0), row32 = __shfl_sync(0xFFFFFFFFu, row[0], 8);
                const bool whole = (follows & 0xFFFFu) == 0xFFFFu && row32 == row0 + 32;
                // rows are needed up to a multiple of 16, the MMA's K
                const bool used = lane < 16 && 4 * lane < ((count + 15) & ~15);
                const bool loads = used && (!box || (lane & 7) == 0);
                const uint32_t z_bytes = whole ? kWgPanel
                                               : 4096u * __popc(__ballot_sync(0xFFFFFFFFu, loads && box)) +
                                                     512u * __popc(__ballot_sync(0xFFFFFFFFu, loads && !box));
                if (it >= static_cast<uint32_t>(slots))
                    ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(empty(s), ((it / slots) & 1u) ^ 1u, err));
                if (!ok) break;
                const uint32_t z = smem_base + s * wa.slot_bytes, bar = full(s);
                if (tc::elect_one()) {
                    tc::mbar_arrive_expect_tx(bar, z_panels * z_bytes + 2 * panels * kWgPanel);
                    if (whole)
                        for (int p = 0; p < z_panels; ++p)
                            tc::tma_load_2d(z + p * kWgPanel, is_a ? &x64 : &y64, col0 + p * 64, row0, bar);
                    const int y = padded + (e0 - first);
                    const uint32_t w = z + kWgCols / 64 * kWgPanel;
                    for (int p = 0; p < panels; ++p) {
                        tc::tma_load_2d(w + p * kWgPanel, is_a ? &map_u : &map_t, p * 64, y, bar);
                        tc::tma_load_2d(w + (panels + p) * kWgPanel, is_a ? &map_u : &map_t, p * 64,
                                        y + static_cast<int>(wa.part_rows), bar);
                    }
                }
                __syncwarp();
                if (!whole && loads) {
                    for (int p = 0; p < z_panels; ++p) {
                        if (box)
                            tc::tma_load_2d(z + p * kWgPanel + lane * 512u, is_a ? &x32 : &y32, col0 + p * 64, row[0], bar);
                        else
                            tc::tma_gather4(z + p * kWgPanel + lane * 512u, is_a ? &x1 : &y1, col0 + p * 64, row, bar);
                    }
                }
                __syncwarp();
                ++it;
                if (++s == slots) s = 0;
            }
        }
        if (lane == 0) {  // every load issued has landed before the block may end
            const uint32_t from = it > static_cast<uint32_t>(slots) ? it - slots : 0u;
            for (uint32_t j = from; j < it; ++j) tc::mbar_wait(full(j % slots), (j / slots) & 1u, err);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMAs
        const uint32_t idesc = tc::idesc_bf16_f32(128, r16, true, true);
        uint32_t it = 0, acc = 0;
        int s = 0;
        bool ok = true;
        const uint64_t z_desc = tc::smem_desc_sw128(smem_base, kWgPanel, 1024u);
        const uint64_t t_desc = tc::smem_desc_sw128(smem_base + kWgCols / 64 * kWgPanel, kWgPanel, 1024u);
        for (int64_t round = 0, unit; (unit = unit_of(round)) < units && ok; ++round) {
            const int adapter = adapter_of(unit);
            int first, last, b0, b1;
            group(adapter, first, last);
            share(last - first, static_cast<int>(unit % wa.splits), b0, b1);
            if (b0 >= b1) continue;  // no tokens: the epilogue writes zeros
            const int e_begin = first + b0 * kWgTok, e_end = min(last, first + b1 * kWgTok);
            const bool me = tc::elect_one();
            const uint32_t i = acc & 1;
            if (me) {
                uint32_t jt = it;
                int js = s;
                ok = tc::mbar_wait(acc_empty(i), ((acc >> 1) & 1u) ^ 1u, err);
                const uint32_t d = tmem + i * kWgUnitCols;
                for (int e0 = e_begin; e0 < e_end && ok; e0 += kWgTok, ++jt) {
                    if (!(ok = tc::mbar_wait(full(js), (jt / slots) & 1u, err))) break;
                    tc::tc_fence_after();
                    const int steps = (min(kWgTok, last - e0) + 15) / 16;
                    const uint32_t off = js * (wa.slot_bytes >> 4);
                    for (int kk = 0; kk < steps; ++kk) {
                        const uint32_t adds = e0 > e_begin || kk > 0;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint64_t zd = z_desc + off + half * (2 * kWgPanel >> 4) + kk * 128u;
                            const uint64_t td = t_desc + off + kk * 128u;
                            tc::mma_f16_ss(d + half * (wa.acc_cols / 2), zd, td, idesc, adds);
                            tc::mma_f16_ss(d + second + half * (wa.acc_cols / 2), zd, td + (panels * kWgPanel >> 4), idesc,
                                           apart ? adds : 1u);
                        }
                    }
                    tc::mma_commit(empty(js));
                    if (++js == slots) js = 0;
                }
                if (ok) tc::mma_commit(acc_full(i));
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, __ffs(__ballot_sync(0xFFFFFFFFu, me)) - 1);
            it += b1 - b0;
            s = it % slots;
            ++acc;
        }
        __syncwarp();
        if (tc::elect_one()) tc::mma_commit(drain);  // every MMA issued has completed before TMEM is released
        __syncwarp();
        tc::mbar_wait(drain, 0u, err);
    } else {
        // ---------------------------------------------------------------- epilogue
        const int w4 = warp & 3;
        uint32_t acc = 0;
        bool ok = true;
        for (int64_t round = 0, unit; (unit = unit_of(round)) < units && ok; ++round) {
            const int sp = static_cast<int>(unit % wa.splits);
            const int adapter = adapter_of(unit);
            const int tile = static_cast<int>(unit / wa.splits % per_adapter);
            const bool is_a = tile < wa.in_tiles;
            const int64_t col0 = static_cast<int64_t>(is_a ? tile : tile - wa.in_tiles) * kWgCols + w4 * 32 + lane;
            const int64_t width = is_a ? g.d_in : g.d_out;
            int first, last, b0, b1;
            group(adapter, first, last);
            share(last - first, sp, b0, b1);
            const bool any = b0 < b1;
            const uint32_t i = acc & 1;
            if (any) {
                ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(acc_full(i), (acc >> 1) & 1u, err));
                if (!ok) break;
                tc::tc_fence_after();
                ++acc;
            }
            for (int half = 0; half < 2; ++half) {
                const int64_t col = col0 + half * 128;
                for (int c0 = 0; c0 < r16; c0 += 32) {
                    uint32_t v[32];
                    if (any) {
                        const uint32_t d = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + i * kWgUnitCols +
                                           half * (wa.acc_cols / 2) + c0;
                        tc::tmem_ld_32x32b_x32(d, v);
                        if (apart) {
                            uint32_t rest[32];
                            tc::tmem_ld_32x32b_x32(d + second, rest);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(join_parts(v[j], rest[j]));
                        } else {
                            tc::tmem_wait_ld();
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                    }
                    if (col >= width) {
                        // past the last column
                    } else if (wa.splits > 1) {
                        float* to = wa.partial + sp * wa.split_stride;
                        if (is_a) {
                            to += (static_cast<int64_t>(adapter) * g.rank + c0) * width + col;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c0 + j < g.rank) to[j * width] = __uint_as_float(v[j]);
                        } else {
                            to += wa.gb_at + (static_cast<int64_t>(adapter) * width + col) * g.rank + c0;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c0 + j < g.rank) to[j] = __uint_as_float(v[j]);
                        }
                    } else if (is_a) {  // neighbouring lanes hold neighbouring columns
                        uint16_t* to = g.gA + (static_cast<int64_t>(adapter) * g.rank + c0) * width + col;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j < g.rank) to[j * width] = float_to_bf16_bits(__uint_as_float(v[j]));
                    } else {
                        uint16_t* to = g.gB + (static_cast<int64_t>(adapter) * width + col) * g.rank + c0;
                        if (g.rank % 8 == 0) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8)
                                if (c0 + j < g.rank)
                                    *reinterpret_cast<uint4*>(to + j) =
                                        make_uint4(pack_bf16(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                                                   pack_bf16(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])),
                                                   pack_bf16(__uint_as_float(v[j + 4]), __uint_as_float(v[j + 5])),
                                                   pack_bf16(__uint_as_float(v[j + 6]), __uint_as_float(v[j + 7])));
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c0 + j < g.rank) to[j] = float_to_bf16_bits(__uint_as_float(v[j]));
                        }
                    }
                    __syncwarp();
                }
            }
            if (any) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(acc_empty(i));
            }
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// gA and gB from the splits' sums, in order, rounded once.
__global__ void __launch_bounds__(256) adapter_wgrad_sum_kernel(const float* partial, int64_t stride, int splits,
                                                                uint16_t* gA, int64_t nA, uint16_t* gB, int64_t nB) {
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < nA + nB; e += static_cast<int64_t>(gridDim.x) * 256) {
        float s = 0.f;
        for (int k = 0; k < splits; ++k) s += partial[k * stride + e];
        (e < nA ? gA[e] : gB[e - nA]) = float_to_bf16_bits(s);
    }
}

}  // namespace nq

// Blocks that share the tokens of a unit: as many as the multiprocessors have room for where the units
// are few, with 512 tokens of the batch each at least.
int nq_adapter_wgrad_splits(int64_t M, int64_t n, int64_t d_in, int64_t d_out) {
    const int64_t units = n * ((d_in + nq::kWgCols - 1) / nq::kWgCols + (d_out + nq::kWgCols - 1) / nq::kWgCols);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({nq_host::sm_count() / units, M / 512, 8})));
}

// u_parts, t_parts: as AdapterArgs describes them (written by the transposed product's kernel).
nq_status nq_launch_adapter_wgrad_umma(const nq::AdapterGradArgs& g, const uint16_t* u_parts, const uint16_t* t_parts,
                                       int64_t part_rows, int part_ld, float* partial, cudaStream_t stream, bool pdl) {
    nq::AdapterWgradArgs wa{};
    wa.g = g;
    wa.part_rows = part_rows;
    wa.panels = (g.rank + 63) / 64;
    wa.r16 = (g.rank + 15) / 16 * 16;
    wa.in_tiles = g.gA ? static_cast<int>((g.d_in + nq::kWgCols - 1) / nq::kWgCols) : 0;
    wa.out_tiles = g.gB ? static_cast<int>((g.d_out + nq::kWgCols - 1) / nq::kWgCols) : 0;
    wa.acc_cols = static_cast<uint32_t>(wa.panels) * 128u;
    const int64_t nA = g.gA ? static_cast<int64_t>(g.n) * g.rank * g.d_in : 0;
    const int64_t nB = g.gB ? static_cast<int64_t>(g.n) * g.rank * g.d_out : 0;
    wa.splits = nq_adapter_wgrad_splits(g.M, g.n, g.d_in, g.d_out);
    wa.partial = partial;
    wa.split_stride = nA + nB;
    wa.gb_at = nA;
    wa.slot_bytes = (nq::kWgCols / 64 + 2 * wa.panels) * nq::kWgPanel;
    const size_t fixed = 1024 + 384 + (g.n <= nq::kWgGroups ? 12 * static_cast<size_t>(g.n) : 0);  // alignment, barriers and order, bounds
    constexpr size_t kSmemMax = 227 * 1024;
    wa.slots = static_cast<int>(std::min<size_t>(nq::kWgMaxSlots, (kSmemMax - fixed) / wa.slot_bytes));
    const size_t smem = fixed + wa.slots * static_cast<size_t>(wa.slot_bytes);

    CUtensorMap x64, x32, x1, y64, y32, y1, mu, mt;
    const int b64[2] = {64, 64}, b32[2] = {64, 32}, b1[2] = {64, 1};
    // an operand that is not asked for is never loaded: its map describes the other one
    const uint16_t* x = g.gA ? g.x : g.ybar;
    const uint16_t* y = g.gB ? g.ybar : g.x;
    const int64_t xd[2] = {g.gA ? g.d_in : g.d_out, g.M}, yd[2] = {g.gB ? g.d_out : g.d_in, g.M};
    // columns past the rank (in 16s) are not read: the boxes get zeros there
    const int64_t ld = part_ld, pd[2] = {wa.r16, 2 * part_rows};
    if (!nq_host::tmap_bf16(&x64, x, 2, xd, xd, b64) || !nq_host::tmap_bf16(&x32, x, 2, xd, xd, b32) ||
        !nq_host::tmap_bf16(&x1, x, 2, xd, xd, b1) || !nq_host::tmap_bf16(&y64, y, 2, yd, yd, b64) ||
        !nq_host::tmap_bf16(&y32, y, 2, yd, yd, b32) || !nq_host::tmap_bf16(&y1, y, 2, yd, yd, b1) ||
        !nq_host::tmap_bf16(&mu, u_parts, 2, pd, &ld, b64) || !nq_host::tmap_bf16(&mt, t_parts, 2, pd, &ld, b64))
        return NQ_ERR_LAUNCH;

    static std::atomic<bool> attr_done[64];  // per device; setting an attribute twice is harmless
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return NQ_ERR_DEVICE;
    if (!attr_done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(nq::adapter_wgrad_umma_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmemMax)) != cudaSuccess)
            return NQ_ERR_LAUNCH;
        attr_done[dev].store(true, std::memory_order_release);
    }
    const int64_t units = static_cast<int64_t>(wa.in_tiles + wa.out_tiles) * g.n * wa.splits;
    const int grid = static_cast<int>(std::min<int64_t>(units, nq_host::sm_count()));
    void* kargs[] = {&x64, &x32, &x1, &y64, &y32, &y1, &mu, &mt, &wa};
    if (nq_host::launch_pdl(reinterpret_cast<const void*>(nq::adapter_wgrad_umma_kernel), dim3(grid),
                            dim3(nq::kWgThreads), smem, stream, kargs, pdl) != cudaSuccess)
        return NQ_ERR_LAUNCH;
    if (wa.splits == 1) return NQ_OK;
    const float* part = partial;
    uint16_t *gA = g.gA, *gB = g.gB;
    int64_t stride = wa.split_stride, nA_arg = nA, nB_arg = nB;
    int splits = wa.splits;
    void* sargs[] = {&part, &stride, &splits, &gA, &nA_arg, &gB, &nB_arg};
    const int64_t blocks = std::min<int64_t>((nA + nB + 255) / 256, 8 * static_cast<int64_t>(nq_host::sm_count()));
    return nq_host::launch_pdl(reinterpret_cast<const void*>(nq::adapter_wgrad_sum_kernel),
                               dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, sargs, pdl) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}
