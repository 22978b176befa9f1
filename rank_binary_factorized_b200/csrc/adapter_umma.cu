// adapter_umma.cu -- low-rank adapters beside a shared projection, on the tensor cores (tcgen05):
//
//   t[m] = scale_a P_a z[m],   out[m] = base[m] + Q_a t[m]      (a = the adapter of row m)
//   forward: z = x, P = A, Q = B;   transposed: z = ybar, P = B^T, Q = A^T
//
// Bound: z, base and out cross HBM once each (2 bytes each way against 2 rank flops per element), so
// the tensor cores are there to keep the products off the critical path and everything else is
// arranged so that the loads never pause.  One launch does both products:
//
// - A tile is up to 128 rows that share an adapter; the rows may lie anywhere (TMA row gathers).  A
//   cluster of CS blocks takes a tile; a block multiplies every CS-th K-block of 64 in the first
//   product and column block of 64 in the second, so a few tiles still use most SMs.
// - Warp 0 loads, warp 1 issues the MMAs, warps 2..9 are the epilogue.  One ring of slots serves both
//   products (a 128 x 64 tile of z, or of base, and the matching tile of P or Q), so the loads of
//   the second product, and of the cluster's next tile, are in flight while t is put together.
// - The blocks' partial t go to the block that owns the row by bulk copies between their shared memories
//   (plain remote stores of the same took three times as long); it adds them in rank order, scales,
//   writes t and sends its rows to every block as the sum of two bf16 values (16 bits of t: rounding
//   t itself to bf16 would add half a unit of its own to the result), in the layout that the second
//   product's A operand has.  Both parts have t's sign and share the accumulator (accumulators of their
//   own cost the epilogue 8% at 8192 rows of a 70B gate).
// - The epilogue adds the accumulator to the tile of base in registers and stores it from a staging tile
//   of its own, so that a slot is free as soon as it is read.
// Measured (B200): 8192 rows of a 70B gate (8192 -> 28672) at rank 64 198 us, 1.09 GB at 5.5 TB/s, 0.84 of the
// measured copy rate; 5000 rows of 8192 x 8192 at rank 16 50 us (4.9 TB/s); one tile alone 15 to 20 us
// (some 4 us to the first tile's data, 3 us between the products).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "adapter_tc.cuh"

namespace nq {

constexpr int kTok = 128;                  // rows of a tile: the MMA's M
constexpr int kNoneTok = 16;               // rows without an adapter in a tile: only copied
constexpr int kStep = 64;                  // K or N elements of a slot
constexpr uint32_t kTokBytes = kTok * 128; // 128 rows x 64 bf16
constexpr int kEpiWarps = 8;
constexpr int kUmmaThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxSlots = 8;
constexpr uint32_t kAccCol = 128;          // the second product's accumulators, 64 columns each
constexpr uint32_t kTmemColumns = 256;

struct AdapterUmmaArgs {
    AdapterArgs a;
    int slots;
    uint32_t slot_bytes;
    int panels;   // 64-element panels of the rank
    int r16;      // rank rounded up to the MMA's K
};

// Two bf16 values and two fp32 addends, rounded once.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t y, uint32_t lo, uint32_t hi) {
    return pack_bf16(__uint_as_float(y << 16) + __uint_as_float(lo),
                     __uint_as_float(y & 0xFFFF0000u) + __uint_as_float(hi));
}

// Barrier of the epilogue's warps.
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory"); }

// Of `segs` segments of partial t in a cluster of cs blocks (16 / cs groups of rows, rounded up, from each);
// at least a tile of out for every warp of the epilogue.
__host__ __device__ constexpr uint32_t inbox_bytes(int segs, int cs) {
    const uint32_t t = static_cast<uint32_t>(segs * cs * ((16 + cs - 1) / cs)) * 1024u;
    return t > kEpiWarps * 4096u ? t : kEpiWarps * 4096u;
}

template <bool BWD>
__global__ void __launch_bounds__(kUmmaThreads, 1)
    adapter_umma_kernel(const __grid_constant__ CUtensorMap map_z, const __grid_constant__ CUtensorMap map_z32,
                        const __grid_constant__ CUtensorMap map_z1, const __grid_constant__ CUtensorMap map_base,
                        const __grid_constant__ CUtensorMap map_base32, const __grid_constant__ CUtensorMap map_base1,
                        const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_a,
                        const __grid_constant__ CUtensorMap map_b, const AdapterUmmaArgs ua) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const AdapterArgs& a = ua.a;
    const uint32_t smem_base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    const int slots = ua.slots, panels = ua.panels, r16 = ua.r16;
    const uint32_t cs = cluster_nctarank(), q = cluster_ctarank();
    // a block puts together the rows of t in groups 16 q / cs .. 16 (q + 1) / cs of 8
    const int own_first = 16 * static_cast<int>(q) / static_cast<int>(cs);
    const int own_groups = 16 * (static_cast<int>(q) + 1) / static_cast<int>(cs) - own_first, own_rows = 8 * own_groups;
    const uint32_t part_bytes = static_cast<uint32_t>(panels) * kTokBytes;
    const uint32_t t_base = smem_base + slots * ua.slot_bytes;  // [2 parts][panels][128 rows][128 B], swizzled
    // Partial t of the rows that this block owns: [cs blocks][segments of 32 ranks][groups][8 pieces of 4
    // ranks][8 rows], 16 bytes a piece.  What a warp of the epilogue holds of a segment and group, it
    // writes and sends as one run of up to 1 KB.
    const int segs = (r16 + 31) / 32;
    const uint32_t seg_bytes = own_groups * 1024u;
    const uint32_t inbox = t_base + 2 * part_bytes;
    const uint32_t staging = inbox;  // between two tiles' t: the epilogue's tiles of out, 4 KB a warp
    const uint32_t bars = inbox + inbox_bytes(segs, static_cast<int>(cs));
    auto slot_at = [&](int s) { return smem_base + s * ua.slot_bytes; };
    auto full = [&](int s) { return bars + 8u * s; };
    auto free1 = [&](int s) { return bars + 8u * (kMaxSlots + s); };      // first product: its MMAs are done
    auto free2 = [&](int s) { return bars + 8u * (2 * kMaxSlots + s); };  // second: the epilogue is done
    const uint32_t acc1_full = bars + 8u * (3 * kMaxSlots), acc1_empty = acc1_full + 8u;
    auto acc2_full = [&](int i) { return acc1_full + 16u + 8u * i; };
    auto acc2_empty = [&](int i) { return acc1_full + 32u + 8u * i; };
    const uint32_t inbox_full = acc1_full + 48u, t_full = acc1_full + 56u, drain = acc1_full + 64u;
    const uint32_t peers_ready = acc1_full + 72u, tmem_slot = acc1_full + 80u;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned int* err = a.err;
    if (warp == 0) {
        if (lane < slots) {
            tc::mbar_init(full(lane), 1);
            tc::mbar_init(free1(lane), 1);
            tc::mbar_init(free2(lane), 4);
        } else if (lane == 8) {
            tc::mbar_init(acc1_full, 1);
            tc::mbar_init(acc1_empty, kEpiWarps);
            tc::mbar_init(inbox_full, kEpiWarps);
            tc::mbar_init(t_full, 1);
            tc::mbar_init(peers_ready, cs);
            tc::mbar_init(drain, 1);
        } else if (lane == 9 || lane == 10) {
            tc::mbar_init(acc2_full(lane - 9), 1);
            tc::mbar_init(acc2_empty(lane - 9), 4);
        }
        tc::mbar_fence_init();
        __syncwarp();
    } else if (warp == 1) {
        tc::tmem_alloc(tmem_slot, kTmemColumns);
        tc::tmem_relinquish();
    } else if (warp == 2 && tc::elect_one()) {
        tc::tma_prefetch_desc(&map_z);
        tc::tma_prefetch_desc(BWD ? &map_b : &map_a);
        tc::tma_prefetch_desc(&map_base);
        tc::tma_prefetch_desc(BWD ? &map_a : &map_b);
        tc::tma_prefetch_desc(&map_out);
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    // Waited for before another block's barriers are used, by each warp where it can afford to: with
    // one block and no cluster launch, a wait by some of the warps did not return before the others'.
    if (cs > 1) cluster_arrive_relaxed();  // the barriers' own fence orders their set-up
    tc::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem_raw + (tmem_slot - tc::smem_u32(smem_raw)));

    const int kb_all = static_cast<int>((a.K + kStep - 1) / kStep), nb_all = static_cast<int>((a.N + kStep - 1) / kStep);
    // Block q takes every cs-th block of 64 from q on: the cluster reads and writes neighbouring pieces of
    // a row at about the same time (1% faster than a range for each block, at 8192 rows of a 70B gate).
    const int kb_n = (kb_all - static_cast<int>(q) + static_cast<int>(cs) - 1) / static_cast<int>(cs);
    const int nb_n = a.out ? (nb_all - static_cast<int>(q) + static_cast<int>(cs) - 1) / static_cast<int>(cs) : 0;
    auto col_at = [&](int i) { return (i * static_cast<int>(cs) + static_cast<int>(q)) * kStep; };
    const uint32_t w1_bytes = BWD ? panels * 8192u : r16 * 128u;
    const uint32_t w2_bytes = BWD ? r16 * 128u : panels * 8192u;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        uint32_t it = 0, was2 = 0, ph1 = 0, ph2 = 0;  // bit s: slot s's last use and barrier phases
        int s = 0;
        bool ok = true;
        auto next = [&](bool second) {  // waits until slot s may be written
            const uint32_t bit = 1u << s;
            if (it >= static_cast<uint32_t>(slots)) {
                if (was2 & bit) {
                    ok = tc::mbar_wait(free2(s), (ph2 >> s) & 1u, err);
                    ph2 ^= bit;
                } else {
                    ok = tc::mbar_wait(free1(s), (ph1 >> s) & 1u, err);
                    ph1 ^= bit;
                }
            }
            was2 = second ? was2 | bit : was2 & ~bit;
        };
        auto advance = [&] {
            ++it;
            if (++s == slots) s = 0;
        };
        for (int tile = blockIdx.x; ok; tile += gridDim.x) {
            const AdapterTile t = find_tile(a.offsets, a.n, a.M, kTok, kNoneTok, tile, err);
            if (t.adapter < 0) break;
            if (t.adapter >= a.n) continue;
            // lane l holds entries 4 l .. 4 l + 3; eight lanes hold a group of 32 rows, which one TMA
            // box fetches where the rows follow one another and over half of it is wanted (rows past the
            // tile's last reach no output), and row gathers where not; one box takes a whole tile
            int32_t row[4];
            bool follow = true;
            const int first32 = __shfl_sync(0xFFFFFFFFu, 4 * lane < t.count ? a.rows[t.first + 4 * lane] : -1, lane & 24);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = lane * 4 + i;
                const int r = e < t.count ? checked_row(a.rows, t.first + e, a.M, err) : -1;
                follow = follow && (e >= t.count || (r >= 0 && r == first32 + (e & 31)));
                row[i] = r >= 0 ? r : static_cast<int32_t>(a.M);  // past the last row: zeros
            }
            const bool used = 4 * lane < t.count;
            const uint32_t follows = __ballot_sync(0xFFFFFFFFu, follow);
            const bool box = ((follows >> (lane & 24)) & 0xFFu) == 0xFFu && t.count - 4 * (lane & 24) > 16;
            const int32_t tile_row0 = __shfl_sync(0xFFFFFFFFu, row[0], 0);
            const bool whole = t.count > 112 && __all_sync(0xFFFFFFFFu, !used || (box && row[0] == tile_row0 + 4 * lane));
            const bool loads = used && (!box || (lane & 7) == 0);
            const uint32_t z_bytes = 4096u * __popc(__ballot_sync(0xFFFFFFFFu, loads && box)) +
                                     512u * __popc(__ballot_sync(0xFFFFFFFFu, loads && !box));
            const bool boxes = whole || __all_sync(0xFFFFFFFFu, !used || box);
            int32_t row0[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) row0[g] = __shfl_sync(0xFFFFFFFFu, row[0], 8 * g);
            // the tile of P or Q that goes with column block b, by one thread
            auto load_w = [&](auto second, int col, uint32_t w, uint32_t bar) {
                if constexpr (second.value == BWD) {  // A: [rank][64 of d_in]
                    tc::tma_load_3d(w, &map_a, col, 0, t.adapter, bar);
                } else {  // B: [64 of d_out][rank], in panels of 64 ranks
                    tc::tma_load_3d(w, &map_b, 0, col, t.adapter, bar);
                    if (panels > 1) tc::tma_load_3d(w + 8192u, &map_b, 64, col, t.adapter, bar);
                }
            };
            auto load_all = [&](auto second, int blocks) {
                constexpr bool kSecond = second.value;
                const CUtensorMap* box_map = kSecond ? &map_base : &map_z;
                const CUtensorMap* box32_map = kSecond ? &map_base32 : &map_z32;
                const CUtensorMap* row_map = kSecond ? &map_base1 : &map_z1;
                const uint32_t bytes = (whole ? kTokBytes : z_bytes) + (kSecond ? w2_bytes : w1_bytes);
                if (boxes) {
                    const bool me = tc::elect_one();
                    if (me) {
                        for (int b = 0; b < blocks; ++b) {
                            next(kSecond);
                            if (!ok) break;
                            const int col = col_at(b);
                            const uint32_t tok = slot_at(s), bar = full(s);
                            tc::mbar_arrive_expect_tx(bar, bytes);
                            if (whole) {
                                tc::tma_load_2d(tok, box_map, col, tile_row0, bar);
                            } else {
#pragma unroll
                                for (int g = 0; g < 4; ++g)
                                    if (32 * g < t.count)
                                        tc::tma_load_2d(tok + g * 4096u, box32_map, col, row0[g], bar);
                            }
                            load_w(second, col, tok + kTokBytes, bar);
                            advance();
                        }
                    }
                    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, me)) - 1;  // the state goes to every lane
                    it = __shfl_sync(0xFFFFFFFFu, it, src);
                    s = __shfl_sync(0xFFFFFFFFu, s, src);
                    was2 = __shfl_sync(0xFFFFFFFFu, was2, src);
                    ph1 = __shfl_sync(0xFFFFFFFFu, ph1, src);
                    ph2 = __shfl_sync(0xFFFFFFFFu, ph2, src);
                    ok = __shfl_sync(0xFFFFFFFFu, ok, src);
                } else {
                    for (int b = 0; b < blocks; ++b) {
                        next(kSecond);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        const int col = col_at(b);
                        const uint32_t tok = slot_at(s), bar = full(s);
                        if (tc::elect_one()) {
                            tc::mbar_arrive_expect_tx(bar, bytes);
                            load_w(second, col, tok + kTokBytes, bar);
                        }
                        __syncwarp();
                        if (loads) {
                            if (box)
                                tc::tma_load_2d(tok + lane * 512u, box32_map, col, row[0], bar);
                            else
                                tc::tma_gather4(tok + lane * 512u, row_map, col, row, bar);
                        }
                        __syncwarp();
                        advance();
                    }
                }
            };
            load_all(std::false_type{}, kb_n);
            if (ok) load_all(std::true_type{}, nb_n);
        }
        // every load issued has landed before the block may end
        if (lane == 0) {
            const uint32_t first = it > static_cast<uint32_t>(slots) ? it - slots : 0u;
            for (uint32_t j = first; j < it; ++j) tc::mbar_wait(full(j % slots), (j / slots) & 1u, err);
        }
        __syncwarp();
        if (cs > 1) cluster_wait();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMAs
        const uint32_t idesc1 = tc::idesc_bf16_f32(kTok, r16, false, BWD);
        const uint32_t idesc2 = tc::idesc_bf16_f32(kTok, kStep, false, BWD);
        // descriptors of slot 0 and of t; the start address is their lowest field, in 16 bytes
        const uint64_t tok_desc = tc::smem_desc_sw128(smem_base, 16u, 1024u);
        const uint64_t w1_desc = tc::smem_desc_sw128(smem_base + kTokBytes, BWD ? 8192u : 16u, 1024u);
        const uint64_t w2_desc = tc::smem_desc_sw128(smem_base + kTokBytes, BWD ? 8192u : 16u, 1024u);
        const uint64_t t_desc = tc::smem_desc_sw128(t_base, 16u, 1024u);
        uint32_t it = 0, tiles = 0, acc2 = 0;
        int s = 0;
        bool ok = true;
        int tile = blockIdx.x;
        AdapterTile t = find_tile(a.offsets, a.n, a.M, kTok, kNoneTok, tile, err), t_next;
        for (; ok && t.adapter >= 0; t = t_next) {
            tile += gridDim.x;
            t_next = find_tile(a.offsets, a.n, a.M, kTok, kNoneTok, tile, err);
            if (t.adapter >= a.n) continue;
            const bool me = tc::elect_one();
            if (me) {
                uint32_t jt = it, jacc = acc2;
                int js = s;
                if (kb_n > 0) {
                    ok = tc::mbar_wait(acc1_empty, (tiles & 1u) ^ 1u, err);
                    for (int b = 0; b < kb_n && ok; ++b, ++jt) {
                        if (!(ok = tc::mbar_wait(full(js), (jt / slots) & 1u, err))) break;
                        tc::tc_fence_after();
                        const uint32_t off = js * (ua.slot_bytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < kStep / 16; ++kk)
                            tc::mma_f16_ss(tmem, tok_desc + off + kk * 2u, w1_desc + off + kk * (BWD ? 128u : 2u), idesc1,
                                           (b > 0 || kk > 0) ? 1u : 0u);
                        tc::mma_commit(free1(js));
                        if (++js == slots) js = 0;
                    }
                    if (ok) tc::mma_commit(acc1_full);
                }
                if (ok && nb_n > 0) {
                    ok = tc::mbar_wait(t_full, tiles & 1u, err);
                    tc::fence_proxy_async_smem();  // t was written by threads
                    for (int b = 0; b < nb_n && ok; ++b, ++jt, ++jacc) {
                        const uint32_t i = jacc & 1;
                        ok = tc::mbar_wait(full(js), (jt / slots) & 1u, err) &&
                             tc::mbar_wait(acc2_empty(i), ((jacc >> 1) & 1u) ^ 1u, err);
                        if (!ok) break;
                        tc::tc_fence_after();
                        const uint32_t off = js * (ua.slot_bytes >> 4), d = tmem + kAccCol + i * kStep;
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            if (kk * 16 < r16) {
                                const uint64_t td = t_desc + (kk / 4) * (kTokBytes >> 4) + (kk % 4) * 2u;
                                const uint64_t wd = w2_desc + off + (BWD ? kk * 128u : (kk / 4) * 512u + (kk % 4) * 2u);
                                tc::mma_f16_ss(d, td, wd, idesc2, kk > 0 ? 1u : 0u);
                                tc::mma_f16_ss(d, td + (part_bytes >> 4), wd, idesc2, 1u);
                            }
                        }
                        tc::mma_commit(acc2_full(i));
                        if (++js == slots) js = 0;
                    }
                }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, __ffs(__ballot_sync(0xFFFFFFFFu, me)) - 1);
            it += kb_n + nb_n;
            acc2 += nb_n;
            s = it % slots;
            ++tiles;
        }
        __syncwarp();
        if (tc::elect_one()) tc::mma_commit(drain);  // every MMA issued has completed before TMEM is released
        __syncwarp();
        tc::mbar_wait(drain, 0u, err);
        __syncwarp();
        if (cs > 1) cluster_wait();
    } else {
        // ---------------------------------------------------------------- epilogue
        // two sets of four warps take the column blocks in turn
        const int w4 = warp & 3;         // TMEM lanes 32 w4 .. 32 w4 + 31
        const int set = (warp - 2) / 4;
        const int tid = w4 * 32 + lane;  // row of the tile
        const int eid = threadIdx.x - 64;
        uint32_t it = 0, tiles = 0, acc2 = 0;
        int s = 0;
        bool ok = true;
        int tile = blockIdx.x;
        AdapterTile t = find_tile(a.offsets, a.n, a.M, kTok, kNoneTok, tile, err), t_next;
        if (cs > 1) cluster_wait();  // every block's barriers are set up
        // A warp whose wait gave up goes through the remaining tiles without work or waits: the others
        // meet it at the barriers below.
        for (; t.adapter >= 0; t = t_next) {
            tile += gridDim.x;
            t_next = find_tile(a.offsets, a.n, a.M, kTok, kNoneTok, tile, err);
            const int my_row = tid < t.count ? checked_row(a.rows, t.first + tid, a.M, err) : -1;
            if (t.adapter >= a.n) {
                // rows without an adapter: t = 0, out = base (this block's columns)
                if (a.t && q == 0 && set == 0 && my_row >= 0)
                    for (int r = 0; r < a.rank; ++r) a.t[static_cast<int64_t>(my_row) * a.rank + r] = 0.f;
                if (a.out && a.out != a.base) {
                    // 16 rows, pieces of 16 bytes side by side over the epilogue's threads
                    const int64_t c0 = static_cast<int64_t>(nb_all) * q / cs * kStep;
                    const int pieces = static_cast<int>((min(a.N, static_cast<int64_t>(nb_all) * (q + 1) / cs * kStep) - c0) / 8);
                    for (int m0 = 0; m0 < t.count; m0 += 4) {
                        int row[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            row[i] = m0 + i < t.count ? checked_row(a.rows, t.first + m0 + i, a.M, err) : -1;
                        for (int e = eid; e < pieces; e += 32 * kEpiWarps) {
                            uint4 v[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (row[i] >= 0) v[i] = *reinterpret_cast<const uint4*>(a.base + row[i] * a.N + c0 + e * 8);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (row[i] >= 0) *reinterpret_cast<uint4*>(a.out + row[i] * a.N + c0 + e * 8) = v[i];
                        }
                    }
                }
                continue;
            }
            // the 32 rows of this warp: all there and in a row, so that one TMA store takes a box
            const int row0 = __shfl_sync(0xFFFFFFFFu, my_row, 0);
            const bool box = __all_sync(0xFFFFFFFFu, my_row >= 0 && my_row == row0 + lane);
            const float scale = a.scale ? a.scale[t.adapter] : 1.f;
            // ---- this block's share of t, to the rows' owners.  It is put where the owner's rows of t
            // will arrive: t_full of the last tile said that the old t is here, the barrier that every
            // warp is done with it, and peers_ready that every block's inbox is free, which its
            // epilogue has used for tiles of out.
            if (tiles > 0) {
                ok = ok && tc::mbar_wait(t_full, (tiles & 1u) ^ 1u, err);
                if (lane == 0) tc::bulk_wait_group_read<0>();
                tc::fence_proxy_async_smem();  // the writes to the staging tiles before the peers' copies to the inbox
                epilogue_sync();
                if (eid < static_cast<int>(cs)) tc::mbar_arrive_cluster(cluster_map(peers_ready, eid));
                __syncwarp();
                ok = ok && tc::mbar_wait(peers_ready, (tiles & 1u) ^ 1u, err);
            }
            if (ok && kb_n > 0) ok = tc::mbar_wait(acc1_full, tiles & 1u, err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc::tc_fence_after();
            // this lane's group of 8 rows, the block that owns it and its place there
            const int my_group = tid >> 3;
            int owner = my_group * static_cast<int>(cs) / 16;
            if (16 * (owner + 1) / static_cast<int>(cs) <= my_group) ++owner;
            const int owner_first = 16 * owner / static_cast<int>(cs);
            const uint32_t owner_bytes = (16 * (owner + 1) / static_cast<int>(cs) - owner_first) * 1024u;
            const uint32_t at = (my_group - owner_first) * 1024u;
            for (int g = set; g < segs && ok; g += 2) {
                uint32_t v[32];
                if (kb_n > 0) {
                    tc::tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(w4 * 32) << 16) + g * 32, v);
                    tc::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                }
                const int pieces = min(8, (r16 - g * 32) / 4);
                // kept here for this block's own rows, else put where the owner's rows of t will arrive
                const uint32_t home = owner == static_cast<int>(q) ? inbox + (q * segs + g) * seg_bytes + at
                                                                    : t_base + g * kTokBytes + owner_first * 1024u + at;
                uint4* to = reinterpret_cast<uint4*>(smem_raw + (home - tc::smem_u32(smem_raw))) + (lane & 7);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < pieces) to[j * 8] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                tc::fence_proxy_async_smem();
                __syncwarp();
#pragma unroll
                for (int o = 0; o < 32; o += 8) {
                    const int own = __shfl_sync(0xFFFFFFFFu, owner, o);
                    const uint32_t src = __shfl_sync(0xFFFFFFFFu, home, o);
                    const uint32_t off = __shfl_sync(0xFFFFFFFFu, at + (q * segs + g) * owner_bytes, o);
                    if (own != static_cast<int>(q) && tc::elect_one())
                        tc::bulk_copy_cluster(cluster_map(inbox + off, own), src, pieces * 128u, cluster_map(inbox_full, own));
                    __syncwarp();
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kb_n > 0) tc::mbar_arrive(acc1_empty);
                if (eid == 0)
                    tc::mbar_arrive_expect_tx(inbox_full, (cs - 1) * own_rows * r16 * 4u);
                else
                    tc::mbar_arrive(inbox_full);
            }
            // ---- the rows this block owns
            ok = ok && tc::mbar_wait(inbox_full, tiles & 1u, err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            for (int e = eid; e < (r16 / 8) * own_rows && ok; e += 32 * kEpiWarps) {
                const int c = e / own_rows, rr = e - c * own_rows, m = own_first * 8 + rr;
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.f;
                if (m < t.count) {
#pragma unroll 4
                    for (uint32_t src = 0; src < cs; ++src) {
                        const float4* at = reinterpret_cast<const float4*>(
                            smem_raw + (inbox + (src * segs + c / 4) * seg_bytes + (rr >> 3) * 1024u -
                                        tc::smem_u32(smem_raw))) + (rr & 7);
                        const float4 f0 = at[c % 4 * 16], f1 = at[c % 4 * 16 + 8];
                        v[0] += f0.x;
                        v[1] += f0.y;
                        v[2] += f0.z;
                        v[3] += f0.w;
                        v[4] += f1.x;
                        v[5] += f1.y;
                        v[6] += f1.z;
                        v[7] += f1.w;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = c * 8 + j < a.rank ? v[j] * scale : 0.f;
                    if (a.t) {
                        const int row = a.rows[t.first + m];
                        if (row >= 0 && row < a.M) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (c * 8 + j < a.rank) a.t[static_cast<int64_t>(row) * a.rank + c * 8 + j] = v[j];
                        }
                    }
                }
                uint4 hi, lo;
                split_bf16_same_sign(v[0], v[1], hi.x, lo.x);
                split_bf16_same_sign(v[2], v[3], hi.y, lo.y);
                split_bf16_same_sign(v[4], v[5], hi.z, lo.z);
                split_bf16_same_sign(v[6], v[7], hi.w, lo.w);
                uint8_t* at = smem_raw + (t_base - tc::smem_u32(smem_raw)) + (c / 8) * kTokBytes + m * 128 +
                              (((c % 8) ^ (m & 7)) << 4);
                *reinterpret_cast<uint4*>(at) = hi;
                *reinterpret_cast<uint4*>(at + part_bytes) = lo;
                if constexpr (BWD) {
                    if (m < ((t.count + 15) & ~15)) {
                        const int64_t to = (static_cast<int64_t>(t.padded) + m) * a.part_ld + c * 8;
                        const int64_t part = a.part_rows * a.part_ld;
                        if (a.u_parts) {
                            split_for_sums(a.part_ld, v[0], v[1], hi.x, lo.x);
                            split_for_sums(a.part_ld, v[2], v[3], hi.y, lo.y);
                            split_for_sums(a.part_ld, v[4], v[5], hi.z, lo.z);
                            split_for_sums(a.part_ld, v[6], v[7], hi.w, lo.w);
                            *reinterpret_cast<uint4*>(a.u_parts + to) = hi;
                            *reinterpret_cast<uint4*>(a.u_parts + part + to) = lo;
                        }
                        if (a.t_parts) {
                            const int row = m < t.count ? a.rows[t.first + m] : -1;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                v[j] = row >= 0 && row < a.M && c * 8 + j < a.rank
                                           ? a.t_in[static_cast<int64_t>(row) * a.rank + c * 8 + j]
                                           : 0.f;
                            split_for_sums(a.part_ld, v[0], v[1], hi.x, lo.x);
                            split_for_sums(a.part_ld, v[2], v[3], hi.y, lo.y);
                            split_for_sums(a.part_ld, v[4], v[5], hi.z, lo.z);
                            split_for_sums(a.part_ld, v[6], v[7], hi.w, lo.w);
                            *reinterpret_cast<uint4*>(a.t_parts + to) = hi;
                            *reinterpret_cast<uint4*>(a.t_parts + part + to) = lo;
                        }
                    }
                }
            }
            tc::fence_proxy_async_smem();  // the copies and the tensor cores read t
            epilogue_sync();
            if (ok && eid / 32 < static_cast<int>(cs) && static_cast<uint32_t>(eid / 32) != q && tc::elect_one()) {
                const uint32_t bar = cluster_map(t_full, eid / 32);
                for (int g = 0; g < 2 * panels; ++g) {
                    const uint32_t at = t_base + g * kTokBytes + own_first * 1024u;
                    tc::bulk_copy_cluster(cluster_map(at, eid / 32), at, seg_bytes, bar);
                }
            }
            __syncwarp();
            if (eid == 0) tc::mbar_arrive_expect_tx(t_full, (16 - own_groups) * 2 * panels * 1024u);
            // ---- out = base + the second product
            it += kb_n;
            s = it % slots;
            uint8_t* mine = smem_raw + (staging - tc::smem_u32(smem_raw)) + (warp - 2) * 4096;
            for (int b = 0; b < nb_n && ok; ++b, ++acc2) {
                const int i = acc2 & 1;
                if (i != set) {
                    ++it;
                    if (++s == slots) s = 0;
                    continue;
                }
                ok = tc::mbar_wait(full(s), (it / slots) & 1u, err) && tc::mbar_wait(acc2_full(i), (acc2 >> 1) & 1u, err);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc::tc_fence_after();
                uint8_t* tok = smem_raw + (slot_at(s) - tc::smem_u32(smem_raw)) + w4 * 4096;  // 32 rows of 128 bytes
                uint32_t v[64];
                const uint32_t d = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + kAccCol + i * kStep;
                tc::tmem_ld_32x32b_x32(d, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                tc::tmem_ld_32x32b_x32(d + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
                uint4 y[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) y[c] = *reinterpret_cast<const uint4*>(tok + lane * 128 + ((c ^ (lane & 7)) << 4));
                tc::tmem_wait_ld();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(acc2_empty(i));
                    tc::mbar_arrive(free2(s));
                    tc::bulk_wait_group_read<0>();  // this warp's last store has left the staging tile
                }
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    y[c].x = add_bf16x2(y[c].x, v[c * 8], v[c * 8 + 1]);
                    y[c].y = add_bf16x2(y[c].y, v[c * 8 + 2], v[c * 8 + 3]);
                    y[c].z = add_bf16x2(y[c].z, v[c * 8 + 4], v[c * 8 + 5]);
                    y[c].w = add_bf16x2(y[c].w, v[c * 8 + 6], v[c * 8 + 7]);
                    *reinterpret_cast<uint4*>(mine + lane * 128 + ((c ^ (lane & 7)) << 4)) = y[c];
                }
                if (box) {
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tc::tma_store_2d(&map_out, staging + (warp - 2) * 4096u, col_at(b), row0);
                        tc::bulk_commit_group();
                    }
                } else {
                    __syncwarp();
                    // eight lanes store the 128 bytes of a row
                    const int64_t col = col_at(b) + (lane & 7) * 8;
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        y[g] = *reinterpret_cast<const uint4*>(mine + (g * 4 + (lane >> 3)) * 128 +
                                                               (((lane & 7) ^ ((g * 4 + (lane >> 3)) & 7)) << 4));
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        const int row = __shfl_sync(0xFFFFFFFFu, my_row, g * 4 + (lane >> 3));
                        if (row >= 0 && col < a.N)
                            *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(row) * a.N + col) = y[g];
                    }
                    __syncwarp();
                }
                ++it;
                if (++s == slots) s = 0;
            }
            ++tiles;
        }
        // t of the last tile has arrived and the stores have completed before the block ends
        if (tiles > 0) tc::mbar_wait(t_full, (tiles & 1u) ^ 1u, err);
        if (lane == 0) tc::bulk_wait_group<0>();
        __syncwarp();
    }

    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, kTmemColumns);
    }
    if (cs > 1) {  // no block of the cluster writes to this one's shared memory any more
        cluster_arrive();
        cluster_wait();
    }
}

}  // namespace nq

// ------------------------------------------------------------------------------ host side
namespace {

constexpr size_t kUmmaSmemMax = 227 * 1024;

}  // namespace

namespace {

// Clusters of cs blocks of the kernel that fit on the device at once (one block a multiprocessor).
int resident_clusters(int dev, int cs) {
    static std::atomic<int> known[64][9];
    std::atomic<int>& slot = known[dev][cs];
    int n = slot.load(std::memory_order_acquire);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1, static_cast<unsigned>(cs));
        cfg.blockDim = dim3(nq::kUmmaThreads);
        cfg.dynamicSmemBytes = kUmmaSmemMax;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1;
        attr[0].val.clusterDim.y = static_cast<unsigned>(cs);
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, nq::adapter_umma_kernel<false>, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            n = std::max(1, nq_host::sm_count() / (2 * cs));  // unknown: assume half
        }
        slot.store(n, std::memory_order_release);
    }
    return n;
}

}  // namespace

// Every row of z, base, A and B starts on 16 bytes, as TMA needs.
bool nq_adapter_umma_fits(const nq::AdapterArgs& a) {
    return a.K % 8 == 0 && a.N % 8 == 0 && a.lda % 8 == 0 && a.ldb % 8 == 0;
}

nq_status nq_launch_adapter_umma(const nq::AdapterArgs& a, bool backward, cudaStream_t stream, bool pdl) {
    nq::AdapterUmmaArgs ua{};
    ua.a = a;
    ua.r16 = (a.rank + 15) / 16 * 16;
    ua.panels = (a.rank + 63) / 64;
    ua.slot_bytes = nq::kTokBytes + static_cast<uint32_t>(ua.panels) * 8192u;
    CUtensorMap mz, mz32, mz1, mbase, mbase32, mbase1, mout, ma, mb;
    const int box[2] = {64, nq::kTok}, box32[2] = {64, 32}, row_box[2] = {64, 1};
    const int a_box[3] = {64, ua.r16, 1}, b_box[3] = {64, 64, 1};
    const int64_t z_dims[2] = {a.K, a.M}, base_dims[2] = {a.N, a.M};
    const int64_t a_dims[3] = {a.d_in, a.rank, a.n}, a_st[2] = {a.lda, a.lda * a.rank};
    const int64_t b_dims[3] = {a.rank, a.d_out, a.n}, b_st[2] = {a.ldb, a.ldb * a.d_out};
    const bool second = a.out != nullptr;  // without it the second product's maps are not used
    const uint16_t* base = second ? a.base : a.z;
    const uint16_t* out = second ? a.out : a.z;
    const int64_t* bd = second ? base_dims : z_dims;
    if (!nq_host::tmap_bf16(&mz, a.z, 2, z_dims, &a.K, box) || !nq_host::tmap_bf16(&mz32, a.z, 2, z_dims, &a.K, box32) ||
        !nq_host::tmap_bf16(&mz1, a.z, 2, z_dims, &a.K, row_box) || !nq_host::tmap_bf16(&mbase, base, 2, bd, bd, box) ||
        !nq_host::tmap_bf16(&mbase32, base, 2, bd, bd, box32) || !nq_host::tmap_bf16(&mbase1, base, 2, bd, bd, row_box) ||
        !nq_host::tmap_bf16(&mout, out, 2, bd, bd, box32) ||
        !nq_host::tmap_bf16(&ma, a.A, 3, a_dims, a_st, a_box) || !nq_host::tmap_bf16(&mb, a.B, 3, b_dims, b_st, b_box))
        return NQ_ERR_LAUNCH;

    const void* fn = backward ? reinterpret_cast<const void*>(nq::adapter_umma_kernel<true>)
                              : reinterpret_cast<const void*>(nq::adapter_umma_kernel<false>);
    static std::atomic<bool> attr_done[64];  // per device; setting an attribute twice is harmless
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return NQ_ERR_DEVICE;
    if (!attr_done[dev].load(std::memory_order_acquire)) {
        for (const void* f : {reinterpret_cast<const void*>(nq::adapter_umma_kernel<true>),
                              reinterpret_cast<const void*>(nq::adapter_umma_kernel<false>)})
            if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kUmmaSmemMax)) !=
                cudaSuccess)
                return NQ_ERR_LAUNCH;
        attr_done[dev].store(true, std::memory_order_release);
    }
    // The tiles decide how many blocks share one: as many as a portable cluster has while every
    // tile's cluster is resident at once.  How many there are depends on the lists, which only the
    // device has: M / 128 full ones and, for every other group, one that is not.  Clusters loop
    // over what another grouping adds.  Above 64 ranks only powers of two leave room for three slots.
    const int64_t least = (a.M + nq::kTok - 1) / nq::kTok;
    const int64_t most = nq::max_adapter_tiles(a.M, a.n, nq::kTok, nq::kNoneTok);
    const int64_t likely = least + std::min<int64_t>(a.n, a.M) / 2;
    int cs = 8;
    while (cs > 1 && (likely > resident_clusters(dev, cs) || (ua.panels > 1 && (cs & (cs - 1)) != 0))) --cs;
    const size_t fixed = 1024 + 2 * static_cast<size_t>(ua.panels) * nq::kTokBytes +
                         nq::inbox_bytes((ua.r16 + 31) / 32, cs) + 8 * (3 * nq::kMaxSlots) + 88;
    ua.slots = static_cast<int>(std::min<size_t>(nq::kMaxSlots, (kUmmaSmemMax - fixed) / ua.slot_bytes));
    const size_t smem = fixed + ua.slots * static_cast<size_t>(ua.slot_bytes);
    const int64_t clusters = std::min<int64_t>(most, resident_clusters(dev, cs));
    void* kargs[] = {&mz, &mz32, &mz1, &mbase, &mbase32, &mbase1, &mout, &ma, &mb, &ua};
    return nq_host::launch_ex(fn, dim3(static_cast<unsigned>(clusters), static_cast<unsigned>(cs)),
                              dim3(nq::kUmmaThreads), smem, stream, kargs, pdl, cs) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}
