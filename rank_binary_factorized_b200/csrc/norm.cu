// norm.cu -- the norms, gate and residual between two blocks, forward and backward.
//
// For a block output y and the residual stream h of one token (d channels):
//
//   z  = w_post (.) y / q(y)   (post_norm; else z = y),   q(v) = sqrt(mean(v^2) + eps)
//   h' = alpha h + gate (.) z
//   x  = w_pre (.) h' / q(h')                             (the next block's input)
//
// and, with v^ = v / q(v) and c(g, v^) = mean(g v^), for the gradients gh' of h' and gx of x:
//
//   dh' = gh' + (w_pre gx - h'^ c(w_pre gx, h'^)) / q(h'),   g_w_pre  = sum_m gx h'^
//   gh  = alpha dh',   dz = gate dh',   g_gate = dh' z (summed over m for a shared gate)
//   gy  = (w_post dz - y^ c(w_post dz, y^)) / q(y)  (post_norm; else dz),  g_w_post = sum_m dz y^
//
// Everything between the loads and the stores is fp32; each output is rounded once.
//
// Bound: HBM, 6 to 14 bytes an element forward and 12 to 20 backward.  Measured (B200): 16384 rows of 8192
// with an fp32 residual and a gate per row 286 us, 1.88 GB at 6.57 TB/s, the measured copy rate;
// gradients of 8192 x 8192 bf16 135 us and 9 us for the vectors' sums, 0.81 GB at 5.6 TB/s; one row of
// 8192 3.7 us forward, 8.8 us backward.  Rows that do not start on 16 bytes (an odd d) cost the
// arithmetic of the shifts: 16384 x 8191 356 us forward (3.0 TB/s), 616 us backward (2.6 TB/s).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "norm.cuh"
#include "tc_common.cuh"

namespace nq {

__device__ __forceinline__ float ld_h(const void* p, int64_t i, bool f32) {
    return f32 ? static_cast<const float*>(p)[i] : bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void st_h(void* p, int64_t i, bool f32, float v) {
    if (f32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = float_to_bf16_bits(v);
}
__device__ __forceinline__ float ld_w(const uint16_t* w, int64_t i, float offset) {
    return w ? offset + bf16_bits_to_float(w[i]) : 1.0f;
}

constexpr int kNormThreads = 256;

// Sums N values over the block; every thread gets the totals.  Fixed order.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    __syncthreads();  // red may still be read by the previous call
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[warp * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = 0.f;
        for (int w = 0; w < nw; ++w) s += red[w * N + i];
        v[i] = s;
    }
}

// ------------------------------------------------------------------ a thread's share of a row
// A thread holds E elements of a row in pieces of 8 neighbours: piece k starts at column
// (k blockDim + tid) 8.  Where every row starts on 16 bytes (SHIFT false) a piece is one load; else a
// row starts s elements after a 16-byte boundary, the same s for all its pieces, and a piece is cut
// out of the two aligned vectors around it.  Elements past the row's end are 0.
__device__ __forceinline__ int col_of(int k) {
    return (k * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8;
}
__device__ __forceinline__ void unpack8(const uint32_t (&a)[4], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
}
// Elements s .. s + 7 of 16 bf16 (s < 8).
__device__ __forceinline__ void shift16(const uint32_t (&w)[8], uint32_t s, uint32_t (&o)[4]) {
    uint32_t t[6], u[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) t[i] = s & 4u ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) u[i] = s & 2u ? t[i + 1] : t[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __byte_perm(u[i], u[i + 1], s & 1u ? 0x5432u : 0x3210u);
}
// Elements s .. s + 7 of 12 fp32 (s < 4).
__device__ __forceinline__ void shift32(const float (&w)[12], uint32_t s, float (&o)[8]) {
    float t[10];
#pragma unroll
    for (int i = 0; i < 10; ++i) t[i] = s & 2u ? w[i + 2 < 12 ? i + 2 : 11] : w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = s & 1u ? t[i + 1] : t[i];
}
// Eight elements from column c of a row of d; `end`: nothing from there on may be read.
template <bool SHIFT>
__device__ __forceinline__ void load8(const uint16_t* row, int c, int d, const uint16_t* end, float (&v)[8]) {
    uint32_t o[4] = {0u, 0u, 0u, 0u};
    if constexpr (!SHIFT) {
        if (c < d) *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(row + c);
        unpack8(o, v);
    } else {
        const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) >> 1) & 7u;
        const uint16_t* q = row + c - s;
        if (c < d) {
            if (end == nullptr || q + 16 <= end) {
                uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(q);
                if (s) *reinterpret_cast<uint4*>(w + 4) = *reinterpret_cast<const uint4*>(q + 8);
                shift16(w, s, o);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = (c + 2 * i < d ? row[c + 2 * i] : 0u) | (c + 2 * i + 1 < d ? row[c + 2 * i + 1] << 16 : 0u);
            }
        }
        unpack8(o, v);
        if (c + 8 > d) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i >= d) v[i] = 0.f;
        }
    }
}
template <bool SHIFT>
__device__ __forceinline__ void load8(const float* row, int c, int d, const float* end, float (&v)[8]) {
    float w[12];
#pragma unroll
    for (int i = 0; i < 12; ++i) w[i] = 0.f;
    if constexpr (!SHIFT) {
        if (c < d) {
            *reinterpret_cast<float4*>(w) = reinterpret_cast<const float4*>(row + c)[0];
            *reinterpret_cast<float4*>(w + 4) = reinterpret_cast<const float4*>(row + c)[1];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[i];
    } else {
        const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) >> 2) & 3u;
        const float* q = row + c - s;
        if (c < d) {
            if (end == nullptr || q + 12 <= end) {
                *reinterpret_cast<float4*>(w) = reinterpret_cast<const float4*>(q)[0];
                *reinterpret_cast<float4*>(w + 4) = reinterpret_cast<const float4*>(q)[1];
                if (s) *reinterpret_cast<float4*>(w + 8) = reinterpret_cast<const float4*>(q)[2];
            } else {
#pragma unroll
                for (int i = 0; i < 12; ++i)
                    if (i >= static_cast<int>(s) && c + i - static_cast<int>(s) < d) w[i] = q[i];
            }
        }
        shift32(w, s, v);
        if (c + 8 > d) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i >= d) v[i] = 0.f;
        }
    }
}
// A vector of the norm (its start is on 16 bytes, its length need not be).
__device__ __forceinline__ void load8_vector(const uint16_t* w, int c, int d, float (&v)[8]) {
    if (c + 8 <= d) {
        load8<false>(w, c, d, nullptr, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < d ? bf16_bits_to_float(w[c + i]) : 0.f;
    }
}
// Stores a piece.  Where rows are shifted, a lane joins its neighbour's last s elements and its own
// first into aligned vectors; at the ends of a warp and of the row single elements are left.  Every
// lane of the warp calls it.
template <bool SHIFT>
__device__ __forceinline__ void store8(uint16_t* row, int c, int d, const float (&v)[8]) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if constexpr (!SHIFT) {
        if (c < d) *reinterpret_cast<uint4*>(row + c) = make_uint4(p[0], p[1], p[2], p[3]);
    } else {
        const int s = static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1) & 7, lane = threadIdx.x & 31;
        uint32_t w[8], o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __shfl_up_sync(0xFFFFFFFFu, p[i], 1);
            w[4 + i] = p[i];
        }
        if (s == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = p[i];
        } else {
            shift16(w, 8 - s, o);
        }
        if (c < d) {
            if ((lane > 0 || s == 0) && c + 8 - s <= d) {
                *reinterpret_cast<uint4*>(row + c - s) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < 8 - s && c + i < d) row[c + i] = static_cast<uint16_t>(p[i / 2] >> (i % 2 * 16));
            }
            if (lane == 31 || c + 16 - s > d) {  // no neighbour takes the last s
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= 8 - s && c + i < d) row[c + i] = static_cast<uint16_t>(p[i / 2] >> (i % 2 * 16));
            }
        }
    }
}
template <bool SHIFT>
__device__ __forceinline__ void store8(float* row, int c, int d, const float (&v)[8]) {
    if constexpr (!SHIFT) {
        if (c < d) {
            reinterpret_cast<float4*>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
        const int s = static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 2) & 3, lane = threadIdx.x & 31;
        float w[12], o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xFFFFFFFFu, v[4 + i], 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[4 + i] = v[i];
        if (s == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = v[i];
        } else {
            shift32(w, 4 - s, o);
        }
        if (c < d) {
            if ((lane > 0 || s == 0) && c + 8 - s <= d) {
                reinterpret_cast<float4*>(row + c - s)[0] = make_float4(o[0], o[1], o[2], o[3]);
                reinterpret_cast<float4*>(row + c - s)[1] = make_float4(o[4], o[5], o[6], o[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < 8 - s && c + i < d) row[c + i] = v[i];
            }
            if (lane == 31 || c + 16 - s > d) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= 8 - s && c + i < d) row[c + i] = v[i];
            }
        }
    }
}

// Sum over the block, in every thread.  Fixed order; `red` holds 32 floats and may not be in use.
__device__ __forceinline__ float block_sum1(float v, float* red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (nw == 1) return v;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < nw ? red[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Few rows: one block per row, 8 elements a thread, so that a row's loads are all in flight at once and
// what is left is the latency of one load, two reductions and the stores.
template <bool SHIFT, bool F32>
__global__ void __launch_bounds__(1024) block_norm_rows_kernel(const NormFwdArgs a) {
    using H = std::conditional_t<F32, float, uint16_t>;
    __shared__ float red[2][32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t m = blockIdx.x, base = m * a.d;
    const int d = static_cast<int>(a.d), c = col_of(0);
    const int64_t all = static_cast<int64_t>(gridDim.x) * a.d;
    float h[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (a.w_pre) {
        load8_vector(a.w_pre, c, d, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] += a.w_offset;
    }
    load8<SHIFT>(static_cast<const H*>(a.h) + base, c, d, static_cast<const H*>(a.h) + all, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] *= a.alpha;
    if (a.y) {
        float y[8], g[8], wp[8];
        load8<SHIFT>(a.y + base, c, d, a.y + all, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = wp[i] = 1.f;
        if (a.gate && a.ld_gate > 0)
            load8<SHIFT>(a.gate + m * a.ld_gate, c, d, a.gate + (gridDim.x - 1) * a.ld_gate + d, g);
        else if (a.gate)
            load8_vector(a.gate, c, d, g);
        if (a.post) {
            if (a.w_post) {
                load8_vector(a.w_post, c, d, wp);
#pragma unroll
                for (int i = 0; i < 8; ++i) wp[i] += a.w_offset;
            }
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(y[i], y[i], s);
            const float rp = rsqrtf(block_sum1(s, red[0]) / static_cast<float>(d) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= rp * wp[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = fmaf(y[i], g[i], h[i]);
    }
    if (a.h_out) store8<SHIFT>(static_cast<H*>(a.h_out) + base, c, d, h);
    if (a.x) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(h[i], h[i], s);
        const float r = rsqrtf(block_sum1(s, red[1]) / static_cast<float>(d) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] *= r * w[i];
        store8<SHIFT>(a.x + base, c, d, h);
    }
}

// One block per row, three passes over it; any d, any alignment.
__global__ void __launch_bounds__(kNormThreads) block_norm_any_kernel(const NormFwdArgs a) {
    __shared__ float red[32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t m = blockIdx.x, base = m * a.d;
    const uint16_t* gate = a.gate ? a.gate + m * a.ld_gate : nullptr;
    float rp = 1.f;
    if (a.y && a.post) {
        float s[1] = {0.f};
        for (int64_t i = threadIdx.x; i < a.d; i += kNormThreads) {
            const float y = bf16_bits_to_float(a.y[base + i]);
            s[0] = fmaf(y, y, s[0]);
        }
        block_sum(s, red);
        rp = rsqrtf(s[0] / static_cast<float>(a.d) + a.eps);
    }
    auto new_h = [&](int64_t i) {
        float v = a.alpha * ld_h(a.h, base + i, a.h_f32);
        if (a.y) {
            float z = bf16_bits_to_float(a.y[base + i]);
            if (a.post) z = z * rp * ld_w(a.w_post, i, a.w_offset);
            v = gate ? fmaf(bf16_bits_to_float(gate[i]), z, v) : v + z;
        }
        return v;
    };
    float r = 1.f;
    if (a.x) {
        float s[1] = {0.f};
        for (int64_t i = threadIdx.x; i < a.d; i += kNormThreads) {
            const float v = new_h(i);
            s[0] = fmaf(v, v, s[0]);
        }
        block_sum(s, red);
        r = rsqrtf(s[0] / static_cast<float>(a.d) + a.eps);
    }
    for (int64_t i = threadIdx.x; i < a.d; i += kNormThreads) {
        const float v = new_h(i);  // h_out may be h, x may be y: each element is read before it is written
        if (a.h_out) st_h(a.h_out, base + i, a.h_f32, v);
        if (a.x) a.x[base + i] = float_to_bf16_bits(v * r * ld_w(a.w_pre, i, a.w_offset));
    }
}

// Blocks take rows in turn; block b keeps its sums over rows in part[k][b][.], each column always by
// the same thread.
__global__ void __launch_bounds__(kNormThreads) block_norm_grad_any_kernel(const NormBwdArgs a) {
    __shared__ float red[96];
    pdl_wait();
    pdl_launch_dependents();
    const float inv_d = 1.0f / static_cast<float>(a.d);
    const bool row_gate = a.gate && a.ld_gate > 0;
    float* const part0 = a.part[0] ? a.part[0] + static_cast<int64_t>(blockIdx.x) * a.part_ld : nullptr;
    float* const part1 = a.part[1] ? a.part[1] + static_cast<int64_t>(blockIdx.x) * a.part_ld : nullptr;
    for (int64_t i = threadIdx.x; i < a.d; i += kNormThreads) {
        if (part0) part0[i] = 0.f;
        if (part1) part1[i] = 0.f;
    }
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const int64_t base = m * a.d;
        const uint16_t* gate = a.gate ? a.gate + m * a.ld_gate : nullptr;
        float s[3] = {0.f, 0.f, 0.f};
        for (int64_t i = threadIdx.x; i < a.d; i += kNormThreads) {
            const float h = ld_h(a.h_out, base + i, a.h_f32);
            s[0] = fmaf(h, h, s[0]);
            if (a.gx) s[1] = fmaf(ld_w(a.w_pre, i, a.w_offset) * bf16_bits_to_float(a.gx[base + i]), h, s[1]);
            if (a.y && a.post) {
                const float y = bf16_bits_to_float(a.y[base + i]);
                s[2] = fmaf(y, y, s[2]);
            }
        }
        block_sum(s, red);
        const float r = rsqrtf(s[0] * inv_d + a.eps);
        const float c = s[1] * inv_d * r * r;  // mean(w gx h^) / q(h'), for h^ = h' r
        const float rp = a.post ? rsqrtf(s[2] * inv_d + a.eps) : 1.f;
        auto dh_of = [&](int64_t i, float hn) {  // hn = h'^
            float g = a.gh_out ? ld_h(a.gh_out, base + i, a.h_f32) : 0.f;
            if (a.gx) g += r * ld_w(a.w_pre, i, a.w_offset) * bf16_bits_to_float(a.gx[base + i]) - hn * c;
            return g;
        };
        float cp = 0.f;
        if (a.y && a.post) {
            float p[1] = {0.f};
            for (int64_t i = threadIdx.x; i < a.d; i += kNormThreads) {
                float dz = dh_of(i, ld_h(a.h_out, base + i, a.h_f32) * r);
                if (gate) dz *= bf16_bits_to_float(gate[i]);
                p[0] = fmaf(dz * ld_w(a.w_post, i, a.w_offset), bf16_bits_to_float(a.y[base + i]) * rp, p[0]);
            }
            block_sum(p, red);
            cp = p[0] * inv_d;
        }
        for (int64_t i = threadIdx.x; i < a.d; i += kNormThreads) {
            const float hn = ld_h(a.h_out, base + i, a.h_f32) * r;
            const float dh = dh_of(i, hn);
            if (part0 && a.gx) part0[i] += bf16_bits_to_float(a.gx[base + i]) * hn;
            if (a.y) {
                const float gt = gate ? bf16_bits_to_float(gate[i]) : 1.f;
                const float y = bf16_bits_to_float(a.y[base + i]);
                const float w = ld_w(a.w_post, i, a.w_offset);
                const float yn = y * rp, z = a.post ? yn * w : y, dz = dh * gt;
                if (part1) part1[i] += (row_gate ? dz : dh) * yn;
                if (row_gate && a.g_gate_rows) a.g_gate_rows[base + i] = float_to_bf16_bits(dh * z);
                if (a.gy) a.gy[base + i] = float_to_bf16_bits(a.post ? rp * (w * dz - yn * cp) : dz);
            }
            if (a.gh) st_h(a.gh, base + i, a.h_f32, a.alpha * dh);
        }
    }
}

// ------------------------------------------------------------------ rows in shared memory
//
// Many rows: a block takes rows in turn; bulk copies bring them in, a ring of stages ahead of the
// arithmetic, and a thread has 16 columns, whose weights stay in its registers.
constexpr int kRingE = 16;

// What a stage holds of a row, and where: bf16 tensors (y, gx, the gates) and tensors of h's type.
struct NormRing {
    const uint16_t* s16[3];
    const void* sh[2];
    uint32_t off16[3], offh[2];
    uint32_t stage_bytes;
    int stages;
};

// Bytes [from, from + bytes) of `src`, whose `total` bytes start on 16 and whose end need not: the
// copy starts and ends on 16 bytes around them where the tensor allows, the last odd bytes are moved
// by this thread.  Returns the copy's size; element 0 lands at dst + from % 16.
__device__ __forceinline__ uint32_t span_bytes(int64_t from, uint32_t bytes, int64_t total, bool& odd_tail) {
    const int64_t a0 = from & ~int64_t{15};
    int64_t e1 = (from + bytes + 15) & ~int64_t{15};
    odd_tail = e1 > total;
    if (odd_tail) e1 = (from + bytes) & ~int64_t{15};
    return static_cast<uint32_t>(e1 > a0 ? e1 - a0 : 0);
}

// Two fp32 values in one register pair.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo_of(F2 a) { return __uint_as_float(static_cast<uint32_t>(a.v)); }
__device__ __forceinline__ float hi_of(F2 a) { return __uint_as_float(static_cast<uint32_t>(a.v >> 32)); }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Row m into stage s, by one thread.
template <typename H>
__device__ __forceinline__ void load_stage(const NormRing& g, uint8_t* smem, int64_t m, int s, int64_t M, int64_t d,
                                           uint32_t bar) {
    const int64_t f16 = m * d * 2, fh = m * d * static_cast<int64_t>(sizeof(H));
    bool odd16, oddh;
    const uint32_t n16 = span_bytes(f16, static_cast<uint32_t>(d * 2), M * d * 2, odd16);
    const uint32_t nh = span_bytes(fh, static_cast<uint32_t>(d * sizeof(H)), M * d * static_cast<int64_t>(sizeof(H)), oddh);
    uint8_t* st = smem + s * g.stage_bytes;
    uint32_t tx = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) tx += g.s16[i] ? n16 : 0u;
#pragma unroll
    for (int i = 0; i < 2; ++i) tx += g.sh[i] ? nh : 0u;
    if (odd16) {  // next to the tensor's end only
        for (int i = 0; i < 3; ++i)
            if (g.s16[i])
                for (int64_t b = max((f16 + d * 2) & ~int64_t{15}, f16); b < f16 + d * 2; b += 2)
                    *reinterpret_cast<uint16_t*>(st + g.off16[i] + (b - (f16 & ~int64_t{15}))) = g.s16[i][b / 2];
    }
    if (oddh) {
        const int64_t e = fh + d * static_cast<int64_t>(sizeof(H));
        for (int i = 0; i < 2; ++i)
            if (g.sh[i])
                for (int64_t b = max(e & ~int64_t{15}, fh); b < e; b += sizeof(H))
                    *reinterpret_cast<H*>(st + g.offh[i] + (b - (fh & ~int64_t{15}))) =
                        static_cast<const H*>(g.sh[i])[b / static_cast<int64_t>(sizeof(H))];
    }
    tc::mbar_arrive_expect_tx(bar, tx);
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (g.s16[i] && n16)
            tc::bulk_load(tc::smem_u32(st + g.off16[i]), reinterpret_cast<const uint8_t*>(g.s16[i]) + (f16 & ~int64_t{15}),
                          n16, bar);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (g.sh[i] && nh)
            tc::bulk_load(tc::smem_u32(st + g.offh[i]), static_cast<const uint8_t*>(g.sh[i]) + (fh & ~int64_t{15}), nh, bar);
}

// 1, or offset + w, of the piece at column c.
__device__ __forceinline__ void weight8(const uint16_t* w, float offset, int c, int d, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.f;
    if (w) {
        load8_vector(w, c, d, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += offset;
    }
}

// Sum over the block (up to 16 warps), in every thread, with one barrier.  `red` may be reused once
// another barrier has passed.
__device__ __forceinline__ float ring_sum(float v, float* red) {
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (lane & 15) < nw ? red[lane & 15] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

template <typename T, bool SHIFT>
__device__ __forceinline__ void ring_get(const uint8_t* at, bool there, int c, int d, F2 (&v)[4]) {
    float f[8];
    load8<SHIFT>(reinterpret_cast<const T*>(at), c, there ? d : 0, static_cast<const T*>(nullptr), f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
}

// Forward: two reductions a row (of y^2, then of h'^2, which may be far smaller than its two terms:
// it is not expanded into their sums).
template <bool SHIFT, bool F32, bool ROWGATE>
__global__ void __launch_bounds__(512, 1) block_norm_ring_kernel(const NormFwdArgs a, const NormRing ring, int64_t M) {
    using H = std::conditional_t<F32, float, uint16_t>;
    constexpr int P = kRingE / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][16];
    __shared__ __align__(8) uint64_t bar[4];
    const int d = static_cast<int>(a.d);
    const uint32_t bar0 = tc::smem_u32(bar);
    if (threadIdx.x == 0) {
        for (int s = 0; s < ring.stages; ++s) tc::mbar_init(bar0 + 8u * s, 1);
        tc::mbar_fence_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x == 0)
        for (int s = 0; s < ring.stages; ++s)
            if (blockIdx.x + static_cast<int64_t>(s) * gridDim.x < M)
                load_stage<H>(ring, smem, blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s, M, d, bar0 + 8u * s);
    // w_pre' and w_post' times a shared gate, of this thread's columns
    F2 wpre[P][4], wb[P][4];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        float v[8], g[8];
        weight8(a.w_pre, a.w_offset, col_of(k), d, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) wpre[k][i] = f2(v[2 * i], v[2 * i + 1]);
        weight8(a.post ? a.w_post : nullptr, a.w_offset, col_of(k), d, v);
        if (!ROWGATE && a.gate) {
            load8_vector(a.gate, col_of(k), d, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) wb[k][i] = f2(v[2 * i], v[2 * i + 1]);
    }
    const float inv_d = 1.0f / static_cast<float>(d);
    const F2 alpha2 = f2(a.alpha, a.alpha);
    uint32_t it = 0;
    int s = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, ++it) {
        // a wait that gives up leaves stale rows behind; the error word tells
        tc::mbar_wait(bar0 + 8u * s, (it / ring.stages) & 1u, a.err);
        const int64_t base = m * a.d;
        const uint8_t* st16 = smem + s * ring.stage_bytes + (SHIFT ? static_cast<uint32_t>(base * 2) & 15u : 0u);
        const uint8_t* sth = smem + s * ring.stage_bytes + ring.offh[0] +
                             (SHIFT ? static_cast<uint32_t>(base * static_cast<int64_t>(sizeof(H))) & 15u : 0u);
        F2 h[P][4], rp2 = f2(1.f, 1.f);
        if (a.post) {
            F2 sum = f2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                F2 y[4];
                ring_get<uint16_t, SHIFT>(st16, true, col_of(k), d, y);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum = fma2(y[i], y[i], sum);
            }
            const float rp = rsqrtf(ring_sum(lo_of(sum) + hi_of(sum), red[0]) * inv_d + a.eps);
            rp2 = f2(rp, rp);
        }
        F2 sum = f2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            F2 y[4], g[4];
            ring_get<H, SHIFT>(sth, true, col_of(k), d, h[k]);
            ring_get<uint16_t, SHIFT>(st16, a.y != nullptr, col_of(k), d, y);
            if constexpr (ROWGATE) ring_get<uint16_t, SHIFT>(st16 + ring.off16[1], true, col_of(k), d, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                F2 z = wb[k][i] * (y[i] * rp2);
                if constexpr (ROWGATE) z = z * g[i];
                h[k][i] = fma2(alpha2, h[k][i], z);
                sum = fma2(h[k][i], h[k][i], sum);
            }
        }
        // the barrier in here also says that every thread is done with this stage
        const float r = rsqrtf(ring_sum(lo_of(sum) + hi_of(sum), red[1]) * inv_d + a.eps);
        if (threadIdx.x == 0 && m + static_cast<int64_t>(ring.stages) * gridDim.x < M) {
            tc::fence_proxy_async_smem();
            load_stage<H>(ring, smem, m + static_cast<int64_t>(ring.stages) * gridDim.x, s, M, d, bar0 + 8u * s);
        }
        if (!a.post) __syncthreads();  // red[1] is read before the next row writes it
        const F2 r2 = f2(r, r);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            float oh[8], ox[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 x = h[k][i] * (wpre[k][i] * r2);
                oh[2 * i] = lo_of(h[k][i]);
                oh[2 * i + 1] = hi_of(h[k][i]);
                ox[2 * i] = lo_of(x);
                ox[2 * i + 1] = hi_of(x);
            }
            if (a.h_out) store8<SHIFT>(static_cast<H*>(a.h_out) + base, col_of(k), d, oh);
            if (a.x) store8<SHIFT>(a.x + base, col_of(k), d, ox);
        }
        if (++s == ring.stages) s = 0;
    }
}

// Backward: the vectors' gradients are sums over the rows, so a thread keeps its columns' sums in
// registers.  All that a row's gradients need of the whole row are six sums: with
// v = w_pre gx, r = 1 / q(h'), rp = 1 / q(y) and b = w_post gate y,
//   sum h'^2, sum v h', sum y^2, sum b gh', sum b v, sum b h'
// give c = mean(v h'^) / q(h') and, as dh' = gh' + r v - r h' c, also
//   sum w_post dz y = sum b gh' + r sum b v - r c sum b h',
// so that one block-wide reduction a row is enough.  With a shared gate, g_w_post and g_gate are both
// multiples of sum_m dh' y^, column by column, so two sums a column serve three vectors.  At 8192
// channels a multiprocessor has some 4300 cycles a row at HBM's rate, and the arithmetic alone needs
// over half of them: it is done on pairs (two fp32 operations an instruction).
template <bool SHIFT, bool F32, bool ROWGATE>
__global__ void __launch_bounds__(512, 1) block_norm_grad_rows_kernel(const NormBwdArgs a, const NormRing ring) {
    using H = std::conditional_t<F32, float, uint16_t>;
    constexpr int P = kRingE / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][16][8];
    __shared__ __align__(8) uint64_t bar[4];
    const int d = static_cast<int>(a.d), warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const uint32_t bar0 = tc::smem_u32(bar);
    if (threadIdx.x == 0) {
        for (int s = 0; s < ring.stages; ++s) tc::mbar_init(bar0 + 8u * s, 1);
        tc::mbar_fence_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x == 0)
        for (int s = 0; s < ring.stages; ++s)
            if (blockIdx.x + static_cast<int64_t>(s) * gridDim.x < a.M)
                load_stage<H>(ring, smem, blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s, a.M, d, bar0 + 8u * s);

    // w_pre' and w_post' times a shared gate, of this thread's columns
    F2 wpre[P][4], wb[P][4], acc0[P][4], acc1[P][4];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        float v[8], g[8];
        weight8(a.w_pre, a.w_offset, col_of(k), d, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) wpre[k][i] = f2(v[2 * i], v[2 * i + 1]);
        weight8(a.post ? a.w_post : nullptr, a.w_offset, col_of(k), d, v);
        if (!ROWGATE && a.gate) {
            load8_vector(a.gate, col_of(k), d, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wb[k][i] = f2(v[2 * i], v[2 * i + 1]);
            acc0[k][i] = acc1[k][i] = f2(0.f, 0.f);
        }
    }
    const float inv_d = 1.0f / static_cast<float>(d);

    uint32_t it = 0;
    int s = 0;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, ++it) {
        // a wait that gives up leaves stale rows behind; the error word tells
        tc::mbar_wait(bar0 + 8u * s, (it / ring.stages) & 1u, a.err);
        const uint8_t* st = smem + s * ring.stage_bytes;
        const int64_t base = m * a.d;
        const uint32_t lead16 = SHIFT ? static_cast<uint32_t>(base * 2) & 15u : 0u;
        const uint32_t leadh = SHIFT ? static_cast<uint32_t>(base * static_cast<int64_t>(sizeof(H))) & 15u : 0u;
        const uint8_t *py = st + lead16, *pgx = py + ring.off16[1], *pgate = py + ring.off16[2];
        const uint8_t *ph = st + ring.offh[0] + leadh, *pgh = st + ring.offh[1] + leadh;
        F2 part[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) part[k] = f2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            F2 y[4], gx[4], h[4], gh[4], gr[4];
            ring_get<uint16_t, SHIFT>(py, a.y != nullptr, col_of(k), d, y);
            ring_get<uint16_t, SHIFT>(pgx, a.gx != nullptr, col_of(k), d, gx);
            ring_get<H, SHIFT>(ph, true, col_of(k), d, h);
            ring_get<H, SHIFT>(pgh, a.gh_out != nullptr, col_of(k), d, gh);
            if constexpr (ROWGATE) ring_get<uint16_t, SHIFT>(pgate, true, col_of(k), d, gr);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 v = wpre[k][i] * gx[i];
                F2 b = wb[k][i] * y[i];
                if constexpr (ROWGATE) b = b * gr[i];
                part[0] = fma2(h[i], h[i], part[0]);
                part[1] = fma2(v, h[i], part[1]);
                part[2] = fma2(y[i], y[i], part[2]);
                part[3] = fma2(b, gh[i], part[3]);
                part[4] = fma2(b, v, part[4]);
                part[5] = fma2(b, h[i], part[5]);
            }
        }
        // 8 values over 32 lanes, halving the values a lane keeps: lane l ends with value l / 4
        float sum[8];
#pragma unroll
        for (int k = 0; k < 6; ++k) sum[k] = lo_of(part[k]) + hi_of(part[k]);
        sum[6] = sum[7] = 0.f;
#pragma unroll
        for (int w = 4; w >= 1; w /= 2) {
            const bool upper = lane & (4 * w);
#pragma unroll
            for (int k = 0; k < w; ++k) {
                const float keep = upper ? sum[k + w] : sum[k], give = upper ? sum[k] : sum[k + w];
                sum[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 4 * w);
            }
        }
        sum[0] += __shfl_xor_sync(0xFFFFFFFFu, sum[0], 2);
        sum[0] += __shfl_xor_sync(0xFFFFFFFFu, sum[0], 1);
        if ((lane & 3) == 0) red[it & 1][warp][lane >> 2] = sum[0];
        __syncthreads();  // and every thread is done with the last row
        if (threadIdx.x == 0 && it > 0) {
            const int64_t ahead = m + static_cast<int64_t>(ring.stages - 1) * gridDim.x;
            const int ps = s == 0 ? ring.stages - 1 : s - 1;
            if (ahead < a.M) {
                tc::fence_proxy_async_smem();
                load_stage<H>(ring, smem, ahead, ps, a.M, d, bar0 + 8u * ps);
            }
        }
        float all = 0.f;
        for (int w = lane & 3; w < nw; w += 4) all += red[it & 1][w][lane >> 2];
        all += __shfl_xor_sync(0xFFFFFFFFu, all, 1);
        all += __shfl_xor_sync(0xFFFFFFFFu, all, 2);
#pragma unroll
        for (int k = 0; k < 6; ++k) sum[k] = __shfl_sync(0xFFFFFFFFu, all, 4 * k);
        const float r = rsqrtf(sum[0] * inv_d + a.eps);
        const float c = sum[1] * inv_d * r * r;  // mean(v h'^) / q(h')
        const float rp = a.post ? rsqrtf(sum[2] * inv_d + a.eps) : 1.f;
        const float cp = a.post ? (sum[3] + r * sum[4] - r * c * sum[5]) * inv_d * rp : 0.f;  // mean(w_post dz y^)
        const F2 r2 = f2(r, r), nc2 = f2(-c, -c), rp2 = f2(rp, rp), ncp2 = f2(-cp, -cp), alpha2 = f2(a.alpha, a.alpha);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            F2 y[4], gx[4], h[4], gh[4], gr[4];
            ring_get<uint16_t, SHIFT>(py, a.y != nullptr, col_of(k), d, y);
            ring_get<uint16_t, SHIFT>(pgx, a.gx != nullptr, col_of(k), d, gx);
            ring_get<H, SHIFT>(ph, true, col_of(k), d, h);
            ring_get<H, SHIFT>(pgh, a.gh_out != nullptr, col_of(k), d, gh);
            if constexpr (ROWGATE) ring_get<uint16_t, SHIFT>(pgate, true, col_of(k), d, gr);
            float o_y[8], o_h[8], o_g[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 hn = h[i] * r2;
                const F2 dh = fma2(hn, nc2, fma2(wpre[k][i] * gx[i], r2, gh[i]));
                acc0[k][i] = fma2(gx[i], hn, acc0[k][i]);
                const F2 yn = y[i] * rp2;
                F2 b = wb[k][i];
                if constexpr (ROWGATE) {
                    const F2 g = dh * wb[k][i] * yn;  // dh' z
                    o_g[2 * i] = lo_of(g);
                    o_g[2 * i + 1] = hi_of(g);
                    b = b * gr[i];
                    acc1[k][i] = fma2(dh * gr[i], yn, acc1[k][i]);
                } else {
                    acc1[k][i] = fma2(dh, yn, acc1[k][i]);
                }
                const F2 gy = fma2(yn, ncp2, b * dh) * rp2, g = dh * alpha2;
                o_y[2 * i] = lo_of(gy);
                o_y[2 * i + 1] = hi_of(gy);
                o_h[2 * i] = lo_of(g);
                o_h[2 * i + 1] = hi_of(g);
            }
            if (a.gy) store8<SHIFT>(a.gy + base, col_of(k), d, o_y);
            if (a.gh) store8<SHIFT>(static_cast<H*>(a.gh) + base, col_of(k), d, o_h);
            if constexpr (ROWGATE)
                if (a.g_gate_rows) store8<SHIFT>(a.g_gate_rows + base, col_of(k), d, o_g);
        }
        if (++s == ring.stages) s = 0;
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
        if (col_of(k) >= d) continue;
        const int64_t at = static_cast<int64_t>(blockIdx.x) * a.part_ld + col_of(k);  // part_ld: a multiple of 8
        auto put = [&](float* part, const F2 (&v)[4]) {
            float4* to = reinterpret_cast<float4*>(part + at);
            to[0] = make_float4(lo_of(v[0]), hi_of(v[0]), lo_of(v[1]), hi_of(v[1]));
            to[1] = make_float4(lo_of(v[2]), hi_of(v[2]), lo_of(v[3]), hi_of(v[3]));
        };
        if (a.part[0]) put(a.part[0], acc0[k]);
        if (a.part[1]) put(a.part[1], acc1[k]);
    }
}

// The vectors' gradients from the blocks' sums: a block of W warps has 32 C columns (C a lane), a warp
// every W-th block's sums of them, added up in fp64; then the W in order.  Narrow rows come from more
// blocks and have fewer columns: there C = 1 and W = 32 keep more loads in flight.
template <int C, int W>
__global__ void __launch_bounds__(32 * W) norm_vector_sums_kernel(const NormSumArgs a) {
    __shared__ double part[W][32 * C];
    pdl_wait();
    pdl_launch_dependents();
    const bool second = blockIdx.y != 0;
    const float* from = second ? a.part[1] : a.part[0];
    if (!from) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * (32 * C) + lane * C;
    double s[C] = {};
    if (c < a.part_ld) {
#pragma unroll 8
        for (int b = warp; b < a.blocks; b += W) {
            const float* p = from + b * a.part_ld + c;
            if constexpr (C == 4) {
                const float4 v = *reinterpret_cast<const float4*>(p);
                s[0] += v.x;
                s[1] += v.y;
                s[2] += v.z;
                s[3] += v.w;
            } else {
                s[0] += *p;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) part[warp][lane * C + i] = s[i];
    __syncthreads();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (32 * C) + threadIdx.x;
    if (threadIdx.x >= 32 * C || i >= a.d) return;
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += part[w][threadIdx.x];
    const float v = static_cast<float>(sum);
    if (!second) {
        a.g_w_pre[i] = v;
    } else {
        if (a.g_w_post) a.g_w_post[i] = a.gate ? static_cast<float>(sum * bf16_bits_to_float(a.gate[i])) : v;
        if (a.g_gate) a.g_gate[i] = a.w_post ? static_cast<float>(sum * (a.w_offset + bf16_bits_to_float(a.w_post[i]))) : v;
    }
}

}  // namespace nq

namespace {

constexpr size_t kNormSmemMax = 227 * 1024 - 1152;  // and the static part

// Threads for a row of d channels at E elements each.
int row_threads(int64_t d, int E) { return static_cast<int>((d + 32 * E - 1) / (32 * E) * 32); }

constexpr int64_t kRingMaxD = 512 * nq::kRingE;

// Blocks a multiprocessor of the ring kernels: 512 threads with 128 registers each in all.  Shared memory may
// hold fewer of them (backward, fp32 residual, gate per row); the others then run after those.
int ring_blocks_per_sm(int64_t d) { return std::max(1, std::min(16, 512 / row_threads(d, nq::kRingE))); }

// Backward: blocks that share the rows; rows too wide for the ring take two blocks of any size.
int grad_blocks(int64_t d, int64_t M) {
    const int per_sm = d <= kRingMaxD ? ring_blocks_per_sm(d) : 2;
    // narrow rows: some for each block, so that the blocks' sums stay small beside the rows
    const int64_t rows = std::max<int64_t>(1, std::min<int64_t>(4, 2048 / d));
    return static_cast<int>(std::min<int64_t>((M + rows - 1) / rows, static_cast<int64_t>(per_sm) * nq_host::sm_count()));
}

// Lays out the stages: a row that does not start on 16 bytes brings up to 15 before and after it, and
// its last piece is read to the end of a second vector.  False: two stages do not fit.
bool plan_ring(nq::NormRing& g, int64_t d, bool h_f32) {
    uint32_t at = 0;
    auto place = [&](const void* p, size_t elem, uint32_t& off) {
        off = at;
        if (p) at += static_cast<uint32_t>((d * elem + 62 + 127) / 128 * 128);
    };
    for (int i = 0; i < 3; ++i) place(g.s16[i], 2, g.off16[i]);
    for (int i = 0; i < 2; ++i) place(g.sh[i], h_f32 ? 4 : 2, g.offh[i]);
    g.stage_bytes = at;
    const size_t share = kNormSmemMax / ring_blocks_per_sm(d) - 2048;
    g.stages = static_cast<int>(std::max<size_t>(2, std::min<size_t>(4, share / at)));
    return static_cast<size_t>(g.stages) * at <= kNormSmemMax;
}

template <bool SHIFT, bool F32>
const void* ring_kernel(bool row_gate) {
    return row_gate ? reinterpret_cast<const void*>(nq::block_norm_ring_kernel<SHIFT, F32, true>)
                    : reinterpret_cast<const void*>(nq::block_norm_ring_kernel<SHIFT, F32, false>);
}
template <bool SHIFT, bool F32>
const void* grad_kernel(bool row_gate) {
    return row_gate ? reinterpret_cast<const void*>(nq::block_norm_grad_rows_kernel<SHIFT, F32, true>)
                    : reinterpret_cast<const void*>(nq::block_norm_grad_rows_kernel<SHIFT, F32, false>);
}
// The kernel for this alignment, residual type and gate, allowed all of the shared memory (set once per
// device and kernel; setting an attribute twice is harmless).  nullptr: failed.
const void* pick(bool backward, bool shift, bool f32, bool row_gate) {
    const void* fns[2][8] = {{ring_kernel<false, false>(false), ring_kernel<false, false>(true),
                              ring_kernel<false, true>(false), ring_kernel<false, true>(true),
                              ring_kernel<true, false>(false), ring_kernel<true, false>(true),
                              ring_kernel<true, true>(false), ring_kernel<true, true>(true)},
                             {grad_kernel<false, false>(false), grad_kernel<false, false>(true),
                              grad_kernel<false, true>(false), grad_kernel<false, true>(true),
                              grad_kernel<true, false>(false), grad_kernel<true, false>(true),
                              grad_kernel<true, true>(false), grad_kernel<true, true>(true)}};
    const int i = (shift ? 4 : 0) + (f32 ? 2 : 0) + (row_gate ? 1 : 0);
    static std::atomic<bool> done[64][2][8];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return nullptr;
    const void* fn = fns[backward][i];
    if (!done[dev][backward][i].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kNormSmemMax)) !=
            cudaSuccess)
            return nullptr;
        done[dev][backward][i].store(true, std::memory_order_release);
    }
    return fn;
}

nq_status launched(cudaError_t e) { return e == cudaSuccess ? NQ_OK : NQ_ERR_LAUNCH; }

}  // namespace

nq_status nq_launch_block_norm(const nq::NormFwdArgs& a, int64_t M, cudaStream_t stream, bool pdl) {
    nq::NormFwdArgs args = a;
    args.err = nq_host::error_word();
    void* kargs[] = {&args, nullptr, nullptr};
    const bool row_gate = a.gate && a.ld_gate > 0;
    const bool shift = a.d % 8 != 0 || a.ld_gate % 8 != 0;
    // One block per row while about 1000 threads a multiprocessor hold them all at once (3.6 us at 296 rows
    // of 4096 and at 1100 of 1024), the ring above that (5.3 us at 300 and at 1190 rows).
    const bool one_wave = M * row_threads(a.d, 8) <= 1024 * static_cast<int64_t>(nq_host::sm_count());
    if (a.d <= kRingMaxD && !one_wave && !(row_gate && a.ld_gate != a.d)) {
        nq::NormRing ring{};
        ring.s16[0] = a.y;
        ring.s16[1] = row_gate ? a.gate : nullptr;
        ring.sh[0] = a.h;
        if (plan_ring(ring, a.d, a.h_f32)) {
            const void* fn = pick(false, shift, a.h_f32, row_gate);
            if (!fn) return NQ_ERR_LAUNCH;
            kargs[1] = &ring;
            kargs[2] = &M;
            const int64_t blocks = std::min<int64_t>(M, static_cast<int64_t>(ring_blocks_per_sm(a.d)) * nq_host::sm_count());
            return launched(nq_host::launch_pdl(fn, dim3(static_cast<unsigned>(blocks)), dim3(row_threads(a.d, nq::kRingE)),
                                                static_cast<size_t>(ring.stages) * ring.stage_bytes, stream, kargs, pdl));
        }
    }
    const void* fn = reinterpret_cast<const void*>(nq::block_norm_any_kernel);
    int threads = nq::kNormThreads;
    if (a.d <= 8 * 1024) {
        fn = shift ? (a.h_f32 ? reinterpret_cast<const void*>(nq::block_norm_rows_kernel<true, true>)
                              : reinterpret_cast<const void*>(nq::block_norm_rows_kernel<true, false>))
                   : (a.h_f32 ? reinterpret_cast<const void*>(nq::block_norm_rows_kernel<false, true>)
                              : reinterpret_cast<const void*>(nq::block_norm_rows_kernel<false, false>));
        threads = row_threads(a.d, 8);
    }
    return launched(nq_host::launch_pdl(fn, dim3(static_cast<unsigned>(M)), dim3(threads), 0, stream, kargs, pdl));
}

size_t nq_block_norm_grad_ws(int64_t d, int64_t M) {
    return NQ_WS_HEADER_BYTES + 2 * static_cast<size_t>(grad_blocks(d, M)) * ((d + 7) / 8 * 8) * sizeof(float);
}

nq_status nq_launch_block_norm_grad(const nq::NormBwdArgs& a, float* g_w_pre, float* g_w_post, float* g_gate, void* ws,
                                    cudaStream_t stream, bool pdl) {
    const int blocks = grad_blocks(a.d, a.M);
    const bool row_gate = a.gate && a.ld_gate > 0;
    nq::NormBwdArgs args = a;
    args.err = nq_host::error_word();
    args.part_ld = (a.d + 7) / 8 * 8;
    float* p = reinterpret_cast<float*>(static_cast<char*>(ws) + NQ_WS_HEADER_BYTES);
    args.part[0] = g_w_pre ? p : nullptr;
    args.part[1] = g_w_post || g_gate ? p + static_cast<int64_t>(blocks) * args.part_ld : nullptr;
    nq::NormRing ring{};
    ring.s16[0] = a.y;
    ring.s16[1] = a.gx;
    ring.s16[2] = row_gate ? a.gate : nullptr;
    ring.sh[0] = a.h_out;
    ring.sh[1] = a.gh_out;
    const void* fn = reinterpret_cast<const void*>(nq::block_norm_grad_any_kernel);
    int threads = nq::kNormThreads;
    size_t smem = 0;
    if (a.d <= kRingMaxD && !(row_gate && a.ld_gate != a.d) && plan_ring(ring, a.d, a.h_f32)) {
        if (!(fn = pick(true, a.d % 8 != 0, a.h_f32, row_gate))) return NQ_ERR_LAUNCH;
        threads = row_threads(a.d, nq::kRingE);
        smem = static_cast<size_t>(ring.stages) * ring.stage_bytes;
    }
    void* kargs[] = {&args, &ring};
    nq_status st = launched(nq_host::launch_pdl(fn, dim3(blocks), dim3(threads), smem, stream, kargs, pdl));
    if (st != NQ_OK || !(args.part[0] || args.part[1])) return st;
    nq::NormSumArgs sum{};
    sum.part[0] = args.part[0];
    sum.part[1] = args.part[1];
    sum.part_ld = args.part_ld;
    sum.d = a.d;
    sum.blocks = blocks;
    sum.gate = row_gate ? nullptr : a.gate;
    sum.w_post = a.post ? a.w_post : nullptr;
    sum.w_offset = a.w_offset;
    sum.g_w_pre = g_w_pre;
    sum.g_w_post = g_w_post;
    sum.g_gate = g_gate;
    void* sargs[] = {&sum};
    const bool narrow = a.d <= 2048;
    const void* sums = narrow ? reinterpret_cast<const void*>(nq::norm_vector_sums_kernel<1, 32>)
                              : reinterpret_cast<const void*>(nq::norm_vector_sums_kernel<4, 16>);
    const int64_t cols = narrow ? 32 : 128;
    return launched(nq_host::launch_pdl(sums, dim3(static_cast<unsigned>((a.d + cols - 1) / cols), 2),
                                        dim3(narrow ? 1024 : 512), 0, stream, sargs, pdl));
}
