// adapter.cu -- low-rank adapters of many requests beside a shared projection, on the CUDA cores:
// every width, stride and rank, and the small batches.
//
//   t[m] = scale_a A_a x[m],   out[m] = y[m] + B_a t[m]        (a = the adapter of row m)
//   u[m] = scale_a B_a^T ybar[m],   xbar'[m] = xbar[m] + A_a^T u[m]
//   gA_a = sum_m u[m] x[m]^T,   gB_a = sum_m ybar[m] t[m]^T
//
// A decode step is bound by reading A_a and B_a once, and at its smallest by the launch, so one
// launch does both products: a cluster of blocks takes a tile of up to 8 rows that share an
// adapter, each block a slice of the first product's length K and of the second's outputs N.  The
// blocks' partial t meet in distributed shared memory between the two.  Sums are fp32 in a fixed
// order; out is rounded once.
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
    float part[kRowsTile][kMaxRank];  // this block's share of t
    float t[kRowsTile][kMaxRank];     // t, scaled
    float red[kRowsThreads * kRowsTile];
    int row[kRowsTile];
    AdapterTile tile;
};

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
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                const int row = m < count ? s.row[m] : -1;
                for (int k = threadIdx.x * V; k < len; k += kRowsThreads * V) {
                    if constexpr (V == 8) {
                        uint4 w = make_uint4(0u, 0u, 0u, 0u);
                        if (row >= 0) w = *reinterpret_cast<const uint4*>(a.z + row * a.K + k0 + k);
                        *reinterpret_cast<uint4*>(&s.z[m][k]) = w;
                    } else {
                        s.z[m][k] = row >= 0 ? a.z[row * a.K + k0 + k] : static_cast<uint16_t>(0);
                    }
                }
            }
            __syncthreads();
            if constexpr (!BWD) {
                // warp w: t_r for r = w, w + 8, ...; lanes along K
                for (int r = warp; r < R; r += kRowsThreads / 32) {
                    const uint16_t* w = A + r * a.lda + k0;
                    float acc[NT];
#pragma unroll
                    for (int m = 0; m < NT; ++m) acc[m] = 0.f;
#pragma unroll 4
                    for (int k = lane * V; k < len; k += 32 * V) {
                        float wv[V];
                        ld_bf16<V>(w + k, wv);
#pragma unroll
                        for (int m = 0; m < NT; ++m) {
                            float zv[V];
                            ld_bf16<V>(&s.z[m][k], zv);
#pragma unroll
                            for (int i = 0; i < V; ++i) acc[m] = fmaf(wv[i], zv[i], acc[m]);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], o);
                        if (lane == 0) s.part[m][r] += acc[m];  // (m, r) belongs to this warp
                    }
                }
            } else {
                // u_r = sum_k z_k B[k][r]: threads side by side along r, groups of them along K
                const int rv = (R + V - 1) / V;          // vectors of r in a row of B
                const int side = min(rv, kRowsThreads);  // threads along r
                const int groups = kRowsThreads / side;
                const int g = threadIdx.x / side, v0 = threadIdx.x % side;
                for (int vb = 0; vb < rv; vb += side) {
                    const int r0 = (vb + v0) * V;
                    float acc[NT][V];
#pragma unroll
                    for (int m = 0; m < NT; ++m)
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[m][i] = 0.f;
                    if (g < groups && r0 < R) {
#pragma unroll 4
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
                    // the groups' sums meet in shared memory, one row and one element of V at a time
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
#pragma unroll
                        for (int i = 0; i < V; ++i) s.red[threadIdx.x * V + i] = acc[m][i];
                        __syncthreads();
                        for (int e = threadIdx.x; e < side * V; e += kRowsThreads) {
                            const int r = vb * V + e;
                            if (r < R) {
                                float sum = 0.f;
                                for (int gg = 0; gg < groups; ++gg) sum += s.red[gg * side * V + e];
                                s.part[m][r] += sum;
                            }
                        }
                        __syncthreads();
                    }
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
            // out_i = base_i + sum_r B[i][r] t_r: G lanes share a row of B, each with every G-th vector
            const int rv = (R + V - 1) / V;
            int G = 1;
            while (G < rv && G < 32) G *= 2;
            const int gl = lane % G, rows_per_pass = kRowsThreads / G;
            for (int64_t i0 = n_begin; i0 < n_end; i0 += rows_per_pass) {
                const int64_t i = i0 + threadIdx.x / G;
                float acc[NT];
#pragma unroll
                for (int m = 0; m < NT; ++m) acc[m] = 0.f;
                if (i < n_end) {
                    for (int v = gl; v < rv; v += G) {
                        float wv[V];
                        ld_bf16<V>(B + i * a.ldb + v * V, wv);
#pragma unroll
                        for (int m = 0; m < NT; ++m)
#pragma unroll
                            for (int e = 0; e < V; ++e) acc[m] = fmaf(wv[e], s.t[m][v * V + e], acc[m]);
                    }
                }
#pragma unroll
                for (int m = 0; m < NT; ++m)
                    for (int o = G / 2; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], o);
                if (i < n_end) {
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
                        if (m % G == gl && m < count && s.row[m] >= 0) {
                            const int64_t at = s.row[m] * a.N + i;
                            a.out[at] = float_to_bf16_bits(bf16_bits_to_float(a.base[at]) + acc[m]);
                        }
                    }
                }
            }
        } else {
            // out_j = base_j + sum_r u_r A[r][j]: a thread holds V neighbouring j
            for (int64_t j = n_begin + threadIdx.x * V; j < n_end; j += kRowsThreads * V) {
                float acc[NT][V];
#pragma unroll
                for (int m = 0; m < NT; ++m)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[m][i] = 0.f;
#pragma unroll 4
                for (int r = 0; r < R; ++r) {
                    float wv[V];
                    ld_bf16<V>(A + r * a.lda + j, wv);
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
                        const float u = s.t[m][r];
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[m][i] = fmaf(u, wv[i], acc[m][i]);
                    }
                }
#pragma unroll
                for (int m = 0; m < NT; ++m) {
                    if (m < count && s.row[m] >= 0) {
                        const int64_t at = s.row[m] * a.N + j;
                        float bv[V];
                        ld_bf16<V>(a.base + at, bv);
#pragma unroll
                        for (int i = 0; i < V; ++i) a.out[at + i] = float_to_bf16_bits(bv[i] + acc[m][i]);
                    }
                }
            }
        }
    }
    cluster_wait();  // no block of the cluster reads this one's share any more
}

template <bool BWD, int V>
__global__ void __launch_bounds__(kRowsThreads) adapter_rows_kernel(const AdapterArgs a) {
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
            if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(nq::RowsShared)) != cudaSuccess)
                return NQ_ERR_LAUNCH;
        attr_done[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = nq::max_adapter_tiles(a.M, a.n, nq::kRowsTile, nq::kRowsTile);
    // blocks per tile: enough to give every multiprocessor one, at most a portable cluster
    int cs = 8;
    while (cs > 1 && tiles * cs > 2 * static_cast<int64_t>(nq_host::sm_count())) cs /= 2;
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

nq_status nq_launch_adapter_group_rows(const int32_t* ids, int64_t M, int n, int32_t* rows, int32_t* offsets,
                                       cudaStream_t stream, bool pdl) {
    void* kargs[] = {&ids, &M, &n, &rows, &offsets};
    return nq_host::launch_pdl(reinterpret_cast<const void*>(nq::adapter_group_rows_kernel),
                               dim3(static_cast<unsigned>((n + 1 + 7) / 8)), dim3(256), 0, stream, kargs,
                               pdl) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}
