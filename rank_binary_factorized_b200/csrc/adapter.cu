// adapter.cu -- low-rank adapters of many requests beside a shared projection, on the CUDA cores:
// every width, stride and rank, and the small batches.
//
//   t[m] = scale_a A_a x[m],   out[m] = y[m] + B_a t[m]        (a = the adapter of row m)
//   u[m] = scale_a B_a^T ybar[m],   xbar'[m] = xbar[m] + A_a^T u[m]
//   gA_a = sum_m u[m] x[m]^T,   gB_a = sum_m ybar[m] t[m]^T
//
// A decode step is bound by reading A_a and B_a once, and at its smallest by the latency of a launch and
// two dependent reads, so one launch does both products: a cluster of up to 16 blocks takes a tile
// of up to 8 rows that share an adapter, each block a slice of the first product's length K and of
// the second's outputs N, and the blocks' partial t meet in distributed shared memory between the
// two.  Tiles of 8: a decode batch has few rows an adapter, and 8 rows' sums fit the registers.
// Sums are fp32 in a fixed order; out is rounded once.
// Measured (B200, in a CUDA graph): one row of 4096 x 4096 at rank 16 5.7 us, of a 70B gate at rank 64
// 11 us (4.7 MB); 64 rows of 64 adapters at 8192 x 8192, rank 16, 11 us (36.7 MB, 3.3 TB/s).
#include "adapter.cuh"
#include "tc_common.cuh"

namespace nq {

constexpr int kRowsTile = 8;        // rows of a tile
constexpr int kRowsThreads = 256;
constexpr int kRowsChunk = 2048;    // K elements of z kept in shared memory at a time
constexpr int kMaxRank = NQ_ADAPTER_MAX_RANK;

// V consecutive bf16 (16 bytes at V = 8), as fp32.
template <int V>
__device__ __forceinline__ void ld_bf16(const uint16_t* p, float (&v)[V]) {
    if constexpr (V == 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = bf16_bits_to_float(p[i]);
    }
}

struct RowsShared {
    alignas(16) uint16_t z[kRowsTile][kRowsChunk];
    alignas(16) float part[kRowsTile][kMaxRank];  // this block's share of t
    alignas(16) float t[kRowsTile][kMaxRank];     // t, scaled
    float warp_part[kRowsThreads / 32][kRowsTile][kMaxRank];  // BWD: by warp
    int row[kRowsTile];
    AdapterTile tile;
};

// out_i = base_i + sum_r B[i][r] t_r for rows of B of over 32 bytes: G lanes share a row (16 bytes of it
// each at a time), so that a warp reads whole lines, and a lane has G rows' loads in flight.  The
// lanes' sums are exchanged by halves: lane g of the G ends with the sum of its g-th row.
template <int G, int NT>
__device__ __forceinline__ void rows_expand(const AdapterArgs& a, RowsShared& s, const uint16_t* B, int64_t n_begin,
                                            int64_t n_end) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane % G, sub = lane / G, R = a.rank;
    const int count = s.tile.count;
    for (int64_t i0 = n_begin + warp * 32; i0 < n_end; i0 += kRowsThreads) {
        const int64_t mine = i0 + g * (32 / G) + sub, at = min(mine, n_end - 1);
        uint16_t old[NT];
        float acc[NT][G];
#pragma unroll
        for (int m = 0; m < NT; ++m) {
            old[m] = a.base[max(m < count ? s.row[m] : 0, 0) * a.N + at];
#pragma unroll
            for (int j = 0; j < G; ++j) acc[m][j] = 0.f;
        }
        for (int r0 = 0; r0 < R; r0 += 8 * G) {
            const int r = r0 + g * 8;
            uint4 w[G];
#pragma unroll
            for (int j = 0; j < G; ++j)
                w[j] = *reinterpret_cast<const uint4*>(B + min(i0 + j * (32 / G) + sub, n_end - 1) * a.ldb + min(r, R - 8));
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                float t[8];
                *reinterpret_cast<float4*>(t) = *reinterpret_cast<const float4*>(&s.t[m][min(r, R - 8)]);
                *reinterpret_cast<float4*>(t + 4) = *reinterpret_cast<const float4*>(&s.t[m][min(r, R - 8) + 4]);
                if (r >= R) {  // past the rank: counts nothing
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const uint32_t ww[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
                    float sum = acc[m][j];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum = fmaf(__uint_as_float(ww[e] << 16), t[2 * e], sum);
                        sum = fmaf(__uint_as_float(ww[e] & 0xFFFF0000u), t[2 * e + 1], sum);
                    }
                    acc[m][j] = r < R ? sum : acc[m][j];
                }
            }
        }
#pragma unroll
        for (int m = 0; m < NT; ++m) {
#pragma unroll
            for (int o = G / 2; o >= 1; o /= 2) {
                const bool upper = g & o;
#pragma unroll
                for (int j = 0; j < o; ++j) {
                    const float keep = upper ? acc[m][j + o] : acc[m][j], give = upper ? acc[m][j] : acc[m][j + o];
                    acc[m][j] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                }
            }
            if (mine < n_end && m < count && s.row[m] >= 0)
                a.out[s.row[m] * a.N + mine] = float_to_bf16_bits(bf16_bits_to_float(old[m]) + acc[m][0]);
        }
    }
}

// NT rows at most (1, 2, 4 or 8: the loops over rows are unrolled).  V = 8: every row of A, B, z
// and base starts on 16 bytes and every width is a multiple of 8; V = 1: any.
template <bool BWD, int V, int NT>
__device__ __forceinline__ void rows_tile(const AdapterArgs& a, RowsShared& s, uint32_t q, uint32_t nq) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int adapter = s.tile.adapter, count = s.tile.count, R = a.rank;
    const bool none = adapter >= a.n;
    const uint16_t* A = none ? nullptr : a.A + static_cast<int64_t>(adapter) * R * a.lda;
    const uint16_t* B = none ? nullptr : a.B + static_cast<int64_t>(adapter) * a.d_out * a.ldb;

    for (int e = threadIdx.x; e < NT * R; e += kRowsThreads) s.part[e / R][e % R] = 0.f;
    __syncthreads();
    if (!none) {
        const int64_t per = ((a.K + nq - 1) / nq + 7) / 8 * 8;
        const int64_t k_begin = min(a.K, per * q), k_end = min(a.K, k_begin + per);
        for (int64_t k0 = k_begin; k0 < k_end; k0 += kRowsChunk) {
            const int len = static_cast<int>(min(static_cast<int64_t>(kRowsChunk), k_end - k0));
            // rows that are not there read row 0 and count as zeros
            const int vecs = len / V;
#pragma unroll 4
            for (int e = threadIdx.x; e < NT * vecs; e += kRowsThreads) {
                const int m = e / vecs, k = (e - m * vecs) * V, row = m < count ? s.row[m] : -1;
                const uint16_t* from = a.z + max(row, 0) * a.K + k0 + k;
                if constexpr (V == 8) {
                    const uint4 w = *reinterpret_cast<const uint4*>(from);
                    *reinterpret_cast<uint4*>(&s.z[m][k]) = row >= 0 ? w : make_uint4(0u, 0u, 0u, 0u);
                } else {
                    const uint16_t w = *from;
                    s.z[m][k] = row >= 0 ? w : static_cast<uint16_t>(0);
                }
            }
            __syncthreads();
            if constexpr (!BWD) {
                // warp w: t_r for r = w, w + 8, ..., kSide of them at once; lanes along K
                constexpr int kSide = NT <= 2 ? 4 : 2, kWarps = kRowsThreads / 32;
                for (int rb = warp; rb < R; rb += kSide * kWarps) {
                    float acc[kSide][NT];
#pragma unroll
                    for (int j = 0; j < kSide; ++j)
#pragma unroll
                        for (int m = 0; m < NT; ++m) acc[j][m] = 0.f;
#pragma unroll 2
                    for (int k = lane * V; k < len; k += 32 * V) {
                        float wv[kSide][V];
#pragma unroll
                        for (int j = 0; j < kSide; ++j) {
                            const int r = min(rb + j * kWarps, R - 1);  // past the last: read again, not stored
                            ld_bf16<V>(A + r * a.lda + k0 + k, wv[j]);
                        }
#pragma unroll
                        for (int m = 0; m < NT; ++m) {
                            float zv[V];
                            ld_bf16<V>(&s.z[m][k], zv);
#pragma unroll
                            for (int j = 0; j < kSide; ++j)
#pragma unroll
                                for (int i = 0; i < V; ++i) acc[j][m] = fmaf(wv[j][i], zv[i], acc[j][m]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kSide; ++j)
#pragma unroll
                        for (int m = 0; m < NT; ++m) {
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) acc[j][m] += __shfl_xor_sync(0xFFFFFFFFu, acc[j][m], o);
                            const int r = rb + j * kWarps;
                            if (lane == 0 && r < R) s.part[m][r] += acc[j][m];  // (m, r) belongs to this warp
                        }
                }
            } else {
                // u_r = sum_k z_k B[k][r]: `side` lanes (a power of two) side by side along r, the warp's
                // other lanes and the warps along K
                const int rv = (R + V - 1) / V;  // vectors of r in a row of B
                int side = 1;
                while (side < rv && side < 32) side *= 2;
                const int along = 32 / side, g = warp * along + lane / side, groups = kRowsThreads / 32 * along;
                for (int vb = 0; vb < rv; vb += side) {
                    const int r0 = (vb + lane % side) * V;
                    float acc[NT][V];
#pragma unroll
                    for (int m = 0; m < NT; ++m)
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[m][i] = 0.f;
                    if (r0 < R) {
                        constexpr int kUnroll = NT <= 2 ? 8 : 4;
#pragma unroll kUnroll
                        for (int k = g; k < len; k += groups) {
                            float wv[V];
                            ld_bf16<V>(B + (k0 + k) * a.ldb + r0, wv);
#pragma unroll
                            for (int m = 0; m < NT; ++m) {
                                const float zv = bf16_bits_to_float(s.z[m][k]);
#pragma unroll
                                for (int i = 0; i < V; ++i) acc[m][i] = fmaf(zv, wv[i], acc[m][i]);
                            }
                        }
                    }
                    // over the lanes along K; while a lane has several sums, the two of a pair keep half each
                    constexpr int kSums = NT * V;
                    float(&sum)[kSums] = reinterpret_cast<float(&)[kSums]>(acc);
                    int kept = 0;         // index of sum[0]
                    bool writes = true;   // of the lanes that end with the same sum, the lowest
#pragma unroll
                    for (int st = 0; st < 5; ++st) {
                        const int o = 16 >> st, w = kSums >> (st + 1);
                        if (o < side) break;  // the same for every lane
                        const bool upper = lane & o;
                        if (w >= 1) {
#pragma unroll
                            for (int j = 0; j < w; ++j) {
                                const float keep = upper ? sum[j + w] : sum[j], give = upper ? sum[j] : sum[j + w];
                                sum[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                            }
                            kept += upper ? w : 0;
                        } else {
                            sum[0] += __shfl_xor_sync(0xFFFFFFFFu, sum[0], o);
                            writes = writes && !upper;
                        }
                    }
                    const int left = max(1, kSums / along);
#pragma unroll
                    for (int j = 0; j < kSums; ++j) {
                        const int m = (kept + j) / V, i = (kept + j) % V;
                        if (j < left && writes && r0 + i < R) s.warp_part[warp][m][r0 + i] = sum[j];
                    }
                }
                __syncthreads();
                for (int e = threadIdx.x; e < NT * R; e += kRowsThreads) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kRowsThreads / 32; ++w) sum += s.warp_part[w][e / R][e % R];
                    s.part[e / R][e % R] += sum;
                }
            }
            __syncthreads();  // z is rewritten by the next chunk
        }
    }
    __syncthreads();
    // t = scale * the sum of the blocks' shares, in rank order, in every block of the cluster
    cluster_arrive();
    cluster_wait();
    if (!none) {
        const float scale = a.scale ? a.scale[adapter] : 1.f;
        for (int e = threadIdx.x; e < NT * R; e += kRowsThreads) {
            const int m = e / R, r = e % R;
            const uint32_t addr = static_cast<uint32_t>(__cvta_generic_to_shared(&s.part[m][r]));
            float sum = 0.f;
            for (uint32_t c = 0; c < nq; ++c) sum += ld_cluster_f32(cluster_map(addr, c));
            s.t[m][r] = sum * scale;
        }
    }
    cluster_arrive();  // this block has read the others' shares; matched before the block ends
    __syncthreads();
    if (a.t && q == 0) {
        for (int e = threadIdx.x; e < count * R; e += kRowsThreads) {
            const int row = s.row[e / R];
            if (row >= 0) a.t[static_cast<int64_t>(row) * R + e % R] = none ? 0.f : s.t[e / R][e % R];
        }
    }
    if constexpr (BWD) {
        if ((a.u_parts || a.t_parts) && !none && q == 0) {
            // this tile's padded rows; the group's last tile also zeroes those up to a multiple of 16
            const bool last = s.tile.first + count == a.offsets[adapter + 1];
            const int rows = last ? ((s.tile.padded + count + 15) & ~15) - s.tile.padded : kRowsTile;
            const int64_t part = a.part_rows * a.part_ld;
            for (int e = threadIdx.x; e < rows * a.part_ld; e += kRowsThreads) {
                const int m = e / a.part_ld, r = e % a.part_ld;
                const bool there = m < count && r < R;
                const int64_t at = (static_cast<int64_t>(s.tile.padded) + m) * a.part_ld + r;
                auto put = [&](uint16_t* to, float v) {
                    uint32_t hi, lo;
                    split_for_sums(a.part_ld, v, 0.f, hi, lo);
                    to[at] = static_cast<uint16_t>(hi);
                    to[at + part] = static_cast<uint16_t>(lo);
                };
                if (a.u_parts) put(a.u_parts, there ? s.t[m][r] : 0.f);
                if (a.t_parts) {
                    const int row = there ? s.row[m] : -1;
                    put(a.t_parts, row >= 0 ? a.t_in[static_cast<int64_t>(row) * R + r] : 0.f);
                }
            }
        }
    }
    if (a.out && !(none && a.out == a.base)) {
        const int64_t per = ((a.N + nq - 1) / nq + 7) / 8 * 8;
        const int64_t n_begin = min(a.N, per * q), n_end = min(a.N, n_begin + per);
        if (none) {
            for (int m = 0; m < count; ++m) {
                const int row = s.row[m];
                if (row < 0) continue;
                for (int64_t j = n_begin + threadIdx.x * V; j < n_end; j += kRowsThreads * V) {
                    const int64_t at = row * a.N + j;
                    if constexpr (V == 8)
                        *reinterpret_cast<uint4*>(a.out + at) = *reinterpret_cast<const uint4*>(a.base + at);
                    else
                        a.out[at] = a.base[at];
                }
            }
        } else if constexpr (!BWD) {
            if constexpr (V == 8) {
                if (R > 32) {
                    rows_expand<(NT <= 4 ? 8 : 4), NT>(a, s, B, n_begin, n_end);  // registers: G NT sums
                } else if (R > 16) {
                    rows_expand<4, NT>(a, s, B, n_begin, n_end);
                }
            }
            // out_i = base_i + sum_r B[i][r] t_r: a thread has a row of B at a time, kAhead rows' loads in
            // flight; neighbouring threads neighbouring i
            constexpr int kAhead = NT <= 2 ? 4 : 2, kPiece = V == 8 ? 2 : 8;  // vectors of a row loaded at once
            for (int64_t i0 = n_begin + threadIdx.x; (V != 8 || R <= 16) && i0 < n_end; i0 += kAhead * kRowsThreads) {
                float acc[kAhead][NT];
                uint16_t old[kAhead][NT];
#pragma unroll
                for (int h = 0; h < kAhead; ++h)
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
                        const int64_t i = min(i0 + h * kRowsThreads, n_end - 1);
                        acc[h][m] = 0.f;
                        old[h][m] = a.base[max(m < count ? s.row[m] : 0, 0) * a.N + i];
                    }
                for (int r0 = 0; r0 < R; r0 += kPiece * V) {
                    float w[kAhead][kPiece][V];
#pragma unroll
                    for (int h = 0; h < kAhead; ++h)
#pragma unroll
                        for (int v = 0; v < kPiece; ++v) {
                            const int64_t i = min(i0 + h * kRowsThreads, n_end - 1);
                            ld_bf16<V>(B + i * a.ldb + min(r0 + v * V, R - V), w[h][v]);
                        }
#pragma unroll
                    for (int v = 0; v < kPiece; ++v) {
                        if (r0 + v * V >= R) break;  // the same for every thread
#pragma unroll
                        for (int m = 0; m < NT; ++m) {
                            float t[V];
                            if constexpr (V == 8) {
                                *reinterpret_cast<float4*>(t) = *reinterpret_cast<const float4*>(&s.t[m][r0 + v * V]);
                                *reinterpret_cast<float4*>(t + 4) = *reinterpret_cast<const float4*>(&s.t[m][r0 + v * V + 4]);
                            } else {
                                t[0] = s.t[m][r0 + v];
                            }
#pragma unroll
                            for (int e = 0; e < V; ++e)
#pragma unroll
                                for (int h = 0; h < kAhead; ++h) acc[h][m] = fmaf(w[h][v][e], t[e], acc[h][m]);
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < kAhead; ++h)
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
                        const int64_t i = i0 + h * kRowsThreads;
                        if (i < n_end && m < count && s.row[m] >= 0)
                            a.out[s.row[m] * a.N + i] = float_to_bf16_bits(bf16_bits_to_float(old[h][m]) + acc[h][m]);
                    }
            }
        } else {
            // out_j = base_j + sum_r u_r A[r][j]: a thread holds V neighbouring j; where that leaves threads
            // over, groups of threads share the ranks and add up in shared memory
            const int vecs = static_cast<int>((n_end - n_begin + V - 1) / V);
            int share = 1;
            while (V == 8 && share < 8 && 2 * share * vecs <= kRowsThreads) share *= 2;
            const int per = kRowsThreads / share, g = threadIdx.x / per;
            float* sums = &s.warp_part[0][0][0];  // [V][threads]
            for (int v0 = 0; v0 < vecs; v0 += per) {
                const int64_t j = n_begin + static_cast<int64_t>(v0 + threadIdx.x % per) * V;
                const bool in = j < n_end;
                float acc[NT][V];
                alignas(16) uint16_t old[NT][V];
#pragma unroll
                for (int m = 0; m < NT; ++m)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[m][i] = 0.f;
                if (in && g == 0) {
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
                        const uint16_t* from = a.base + max(m < count ? s.row[m] : 0, 0) * a.N + j;
                        if constexpr (V == 8)
                            *reinterpret_cast<uint4*>(old[m]) = *reinterpret_cast<const uint4*>(from);
                        else
                            old[m][0] = *from;
                    }
                }
                if (in) {
                    constexpr int kUnroll = NT <= 2 ? 8 : 4;
#pragma unroll kUnroll
                    for (int r = g; r < R; r += share) {
                        float wv[V];
                        ld_bf16<V>(A + r * a.lda + j, wv);
#pragma unroll
                        for (int m = 0; m < NT; ++m) {
                            const float u = s.t[m][r];
#pragma unroll
                            for (int i = 0; i < V; ++i) acc[m][i] = fmaf(u, wv[i], acc[m][i]);
                        }
                    }
                }
                if (share > 1) {
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
                        __syncthreads();
#pragma unroll
                        for (int i = 0; i < V; ++i) sums[i * kRowsThreads + threadIdx.x] = acc[m][i];
                        __syncthreads();
                        if (g == 0)
                            for (int h = 1; h < share; ++h)
#pragma unroll
                                for (int i = 0; i < V; ++i) acc[m][i] += sums[i * kRowsThreads + h * per + threadIdx.x];
                    }
                }
                if (in && g == 0) {
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
                        if (m < count && s.row[m] >= 0) {
                            uint16_t* to = a.out + s.row[m] * a.N + j;
                            float now[V];
#pragma unroll
                            for (int i = 0; i < V; ++i) now[i] = bf16_bits_to_float(old[m][i]) + acc[m][i];
                            if constexpr (V == 8)
                                *reinterpret_cast<uint4*>(to) =
                                    make_uint4(pack_bf16(now[0], now[1]), pack_bf16(now[2], now[3]),
                                               pack_bf16(now[4], now[5]), pack_bf16(now[6], now[7]));
                            else
                                *to = float_to_bf16_bits(now[0]);
                        }
                    }
                }
            }
        }
    }
    cluster_wait();  // no block of the cluster reads this one's share any more
}

template <bool BWD, int V>
__global__ void __launch_bounds__(kRowsThreads, 2) adapter_rows_kernel(const AdapterArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    RowsShared& s = *reinterpret_cast<RowsShared*>(smem_raw);
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x < 32) {
        const AdapterTile t = find_tile(a.offsets, a.n, a.M, kRowsTile, kRowsTile, static_cast<int>(blockIdx.x),
                                        a.err);
        if (threadIdx.x == 0) s.tile = t;
        if (threadIdx.x < kRowsTile)
            s.row[threadIdx.x] = static_cast<int>(threadIdx.x) < t.count
                                     ? checked_row(a.rows, t.first + threadIdx.x, a.M, a.err)
                                     : -1;
    }
    __syncthreads();
    if (s.tile.adapter < 0) return;  // the same in every block of the cluster
    const uint32_t q = cluster_ctarank(), nq = cluster_nctarank();
    if (s.tile.count <= 1)
        rows_tile<BWD, V, 1>(a, s, q, nq);
    else if (s.tile.count <= 2)
        rows_tile<BWD, V, 2>(a, s, q, nq);
    else if (s.tile.count <= 4)
        rows_tile<BWD, V, 4>(a, s, q, nq);
    else
        rows_tile<BWD, V, 8>(a, s, q, nq);
}

// ------------------------------------------------------------------ gradients of A and B
constexpr int kGradCols = 64;    // columns of x or ybar of a block
constexpr int kGradTokens = 16;  // tokens in shared memory at a time

// Block: 64 columns of x (blockIdx.x < tiles of d_in) or of ybar, one adapter (blockIdx.y).
// Thread: one column, every fourth r.
__global__ void __launch_bounds__(256) adapter_grad_any_kernel(const AdapterGradArgs a) {
    __shared__ float zs[kGradTokens][kGradCols];
    __shared__ float ts[kGradTokens][kMaxRank];
    __shared__ int row[kGradTokens];
    pdl_wait();
    pdl_launch_dependents();
    const int in_tiles = a.gA ? static_cast<int>((a.d_in + kGradCols - 1) / kGradCols) : 0;
    const bool is_a = static_cast<int>(blockIdx.x) < in_tiles;
    const int64_t c0 = static_cast<int64_t>(is_a ? blockIdx.x : blockIdx.x - in_tiles) * kGradCols;
    const uint16_t* z = is_a ? a.x : a.ybar;
    const float* t = is_a ? a.u : a.t;
    const int64_t width = is_a ? a.d_in : a.d_out;
    const int adapter = blockIdx.y, R = a.rank;
    int first, last;
    adapter_bounds(a.offsets, a.n, a.M, adapter, first, last, a.err);
    const int c = threadIdx.x % kGradCols, r0 = threadIdx.x / kGradCols;
    float acc[kMaxRank / 4];
#pragma unroll
    for (int i = 0; i < kMaxRank / 4; ++i) acc[i] = 0.f;
    for (int e0 = first; e0 < last; e0 += kGradTokens) {
        __syncthreads();
        if (threadIdx.x < kGradTokens)
            row[threadIdx.x] = e0 + static_cast<int>(threadIdx.x) < last
                                   ? checked_row(a.rows, e0 + threadIdx.x, a.M, a.err)
                                   : -1;
        __syncthreads();
        for (int e = threadIdx.x; e < kGradTokens * kGradCols; e += 256) {
            const int m = e / kGradCols, cc = e % kGradCols;
            zs[m][cc] = row[m] >= 0 && c0 + cc < width ? bf16_bits_to_float(z[row[m] * width + c0 + cc]) : 0.f;
        }
        for (int e = threadIdx.x; e < kGradTokens * R; e += 256) {
            const int m = e / R, r = e % R;
            ts[m][r] = row[m] >= 0 ? t[static_cast<int64_t>(row[m]) * R + r] : 0.f;
        }
        __syncthreads();
        for (int m = 0; m < kGradTokens; ++m) {
            const float zv = zs[m][c];
#pragma unroll
            for (int i = 0; i < kMaxRank / 4; ++i)
                if (r0 + 4 * i < R) acc[i] = fmaf(zv, ts[m][r0 + 4 * i], acc[i]);
        }
    }
    if (c0 + c < width) {
#pragma unroll
        for (int i = 0; i < kMaxRank / 4; ++i) {
            const int r = r0 + 4 * i;
            if (r >= R) break;
            if (is_a)
                a.gA[(static_cast<int64_t>(adapter) * R + r) * width + c0 + c] = float_to_bf16_bits(acc[i]);
            else
                a.gB[(static_cast<int64_t>(adapter) * width + c0 + c) * R + r] = float_to_bf16_bits(acc[i]);
        }
    }
}

// Few rows an adapter: bound by writing gA and gB, 16 bytes a thread at a time, neighbouring threads side
// by side.  A block has one adapter and either 8 ranks of 2048 columns of gA or a run of gB, and takes the tokens
// 8 at a time.  Widths and rank in multiples of 8.
// Measured: 64 adapters of 8192 x 8192 at rank 16 (33.5 MB of gradients) 18 us after u is there.
constexpr int kSmallTokens = 8;
constexpr int kSmallRanks = 8;    // ranks of gA of a block
constexpr int kSmallPieces = 4;   // 16-byte pieces of gB of a thread

__global__ void __launch_bounds__(256) adapter_grad_small_kernel(const AdapterGradArgs a, int a_tiles, int a_blocks) {
    __shared__ int row[kSmallTokens];
    __shared__ float ts[kSmallTokens][kMaxRank];
    pdl_wait();
    pdl_launch_dependents();
    const int adapter = blockIdx.y, R = a.rank, blk = blockIdx.x;
    const bool is_a = blk < a_blocks;
    int first, last;
    adapter_bounds(a.offsets, a.n, a.M, adapter, first, last, a.err);
    const float* t = is_a ? a.u : a.t;
    auto pack = [](const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    // tokens e0 .. of the group: their rows and t
    auto stage = [&](int e0) {
        __syncthreads();
        if (threadIdx.x < kSmallTokens)
            row[threadIdx.x] = e0 + static_cast<int>(threadIdx.x) < last ? checked_row(a.rows, e0 + threadIdx.x, a.M, a.err)
                                                                          : -1;
        __syncthreads();
        for (int e = threadIdx.x; e < kSmallTokens * R; e += 256) {
            const int m = e / R, r = e - m * R;
            ts[m][r] = row[m] >= 0 ? t[static_cast<int64_t>(row[m]) * R + r] : 0.f;
        }
        __syncthreads();
    };
    if (is_a) {
        const int64_t j = (static_cast<int64_t>(blk % a_tiles) * 256 + threadIdx.x) * 8;
        const int r0 = blk / a_tiles * kSmallRanks;
        const bool in = j < a.d_in;
        float acc[kSmallRanks][8];
#pragma unroll
        for (int r = 0; r < kSmallRanks; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[r][i] = 0.f;
        for (int e0 = first; e0 < last; e0 += kSmallTokens) {
            stage(e0);
            const int count = min(kSmallTokens, last - e0);
#pragma unroll 4
            for (int m = 0; m < count; ++m) {
                if (row[m] < 0 || !in) continue;
                float x[8];
                ld_bf16<8>(a.x + row[m] * a.d_in + j, x);
#pragma unroll
                for (int r = 0; r < kSmallRanks; ++r)
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[r][i] = fmaf(ts[m][r0 + r], x[i], acc[r][i]);
            }
        }
        if (!in) return;
#pragma unroll
        for (int r = 0; r < kSmallRanks; ++r)
            *reinterpret_cast<uint4*>(a.gA + (static_cast<int64_t>(adapter) * R + r0 + r) * a.d_in + j) = pack(acc[r]);
    } else {
        const int per = R / 8;  // pieces of a row of gB
        const int64_t pieces = a.d_out * per, p0 = static_cast<int64_t>(blk - a_blocks) * (256 * kSmallPieces) + threadIdx.x;
        float acc[kSmallPieces][8];
#pragma unroll
        for (int k = 0; k < kSmallPieces; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[k][i] = 0.f;
        for (int e0 = first; e0 < last; e0 += kSmallTokens) {
            stage(e0);
            const int count = min(kSmallTokens, last - e0);
#pragma unroll
            for (int k = 0; k < kSmallPieces; ++k) {
                const int64_t p = min(p0 + k * 256, pieces - 1), i0 = p / per;
                const int r = static_cast<int>(p - i0 * per) * 8;
#pragma unroll 4
                for (int m = 0; m < count; ++m) {
                    if (row[m] < 0) continue;
                    const float y = bf16_bits_to_float(a.ybar[row[m] * a.d_out + i0]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[k][i] = fmaf(y, ts[m][r + i], acc[k][i]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kSmallPieces; ++k)
            if (p0 + k * 256 < pieces)
                *reinterpret_cast<uint4*>(a.gB + static_cast<int64_t>(adapter) * a.d_out * R + (p0 + k * 256) * 8) = pack(acc[k]);
    }
}

// ------------------------------------------------------------------ rows grouped by adapter
// One warp per group (adapter, then the rows without one): it counts the rows of the groups before
// its own, then writes its own rows in order.  No atomics: the order is that of the rows.
__global__ void __launch_bounds__(256) adapter_group_rows_kernel(const int32_t* ids, int64_t M, int n, int32_t* rows,
                                                                 int32_t* offsets) {
    pdl_wait();
    pdl_launch_dependents();
    const int g = static_cast<int>(blockIdx.x) * (256 / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (g > n) return;
    auto group = [&](int64_t m) {
        const int id = ids[m];
        return id >= 0 && id < n ? id : n;
    };
    int before = 0;
    for (int64_t m = lane; m < M; m += 32) before += group(m) < g;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    if (lane == 0) offsets[g] = before;
    for (int64_t m0 = 0; m0 < M; m0 += 32) {
        const bool mine = m0 + lane < M && group(m0 + lane) == g;
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, mine);
        if (mine) rows[before + __popc(hit & ((1u << lane) - 1u))] = static_cast<int32_t>(m0 + lane);
        before += __popc(hit);
    }
}

}  // namespace nq

// ------------------------------------------------------------------------------ host side
#include <algorithm>
#include <atomic>

namespace {

// Every row of the operands starts on 16 bytes and every width is a multiple of 8 elements.
bool rows_vectors(const nq::AdapterArgs& a) {
    return a.K % 8 == 0 && a.N % 8 == 0 && a.lda % 8 == 0 && a.ldb % 8 == 0 && a.rank % 8 == 0;
}

}  // namespace

nq_status nq_launch_adapter_rows(const nq::AdapterArgs& a, bool backward, cudaStream_t stream, bool pdl) {
    nq::AdapterArgs args = a;
    const bool vec = rows_vectors(a);
    const void* fns[4] = {reinterpret_cast<const void*>(nq::adapter_rows_kernel<false, 1>),
                          reinterpret_cast<const void*>(nq::adapter_rows_kernel<false, 8>),
                          reinterpret_cast<const void*>(nq::adapter_rows_kernel<true, 1>),
                          reinterpret_cast<const void*>(nq::adapter_rows_kernel<true, 8>)};
    static std::atomic<bool> attr_done[64];  // per device; setting an attribute twice is harmless
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return NQ_ERR_DEVICE;
    if (!attr_done[dev].load(std::memory_order_acquire)) {
        for (const void* f : fns)
            if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(nq::RowsShared)) != cudaSuccess ||
                cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
                return NQ_ERR_LAUNCH;
        attr_done[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = nq::max_adapter_tiles(a.M, a.n, nq::kRowsTile, nq::kRowsTile);
    // blocks per tile: what two blocks a multiprocessor have room for, 16 at most (a cluster of 16 needs
    // the multiprocessors of one GPC: only where the tiles are few)
    const int64_t sms = nq_host::sm_count();
    int cs = 16;
    if (tiles * cs > sms / 2) cs = 8;
    while (cs > 1 && tiles * cs > 2 * sms) cs /= 2;
    void* kargs[] = {&args};
    return nq_host::launch_ex(fns[(backward ? 2 : 0) + (vec ? 1 : 0)],
                              dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(cs)), dim3(nq::kRowsThreads),
                              sizeof(nq::RowsShared), stream, kargs, pdl, cs) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}

nq_status nq_launch_adapter_grad_any(const nq::AdapterGradArgs& a, cudaStream_t stream, bool pdl) {
    nq::AdapterGradArgs args = a;
    int64_t tiles = 0;
    if (a.gA) tiles += (a.d_in + nq::kGradCols - 1) / nq::kGradCols;
    if (a.gB) tiles += (a.d_out + nq::kGradCols - 1) / nq::kGradCols;
    if (tiles == 0) return NQ_OK;
    void* kargs[] = {&args};
    return nq_host::launch_pdl(reinterpret_cast<const void*>(nq::adapter_grad_any_kernel),
                               dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(a.n)), dim3(256), 0, stream,
                               kargs, pdl) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}

nq_status nq_launch_adapter_grad_small(const nq::AdapterGradArgs& a, cudaStream_t stream, bool pdl) {
    nq::AdapterGradArgs args = a;
    int a_tiles = static_cast<int>((a.d_in + 2047) / 2048);
    int a_blocks = a.gA ? a_tiles * (a.rank / nq::kSmallRanks) : 0;
    const int64_t b_blocks =
        a.gB ? (a.d_out * (a.rank / 8) + 256 * nq::kSmallPieces - 1) / (256 * nq::kSmallPieces) : 0;
    void* kargs[] = {&args, &a_tiles, &a_blocks};
    return nq_host::launch_pdl(reinterpret_cast<const void*>(nq::adapter_grad_small_kernel),
                               dim3(static_cast<unsigned>(a_blocks + b_blocks), static_cast<unsigned>(a.n)), dim3(256), 0,
                               stream, kargs, pdl) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}

nq_status nq_launch_adapter_group_rows(const int32_t* ids, int64_t M, int n, int32_t* rows, int32_t* offsets,
                                       cudaStream_t stream, bool pdl) {
    void* kargs[] = {&ids, &M, &n, &rows, &offsets};
    return nq_host::launch_pdl(reinterpret_cast<const void*>(nq::adapter_group_rows_kernel),
                               dim3(static_cast<unsigned>((n + 1 + 7) / 8)), dim3(256), 0, stream, kargs,
                               pdl) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}
