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
// E elements of a row in a block of T threads.  VEC: pieces of 8 neighbours (16 bytes of bf16), the
// row starts on 16 bytes; else single elements, neighbouring threads side by side.
template <bool VEC>
__device__ __forceinline__ int col_of(int e) {
    return VEC ? ((e / 8) * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8 + e % 8
               : e * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
}
__device__ __forceinline__ void unpack8(const uint4 w, float* v) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return static_cast<uint32_t>(float_to_bf16_bits(lo)) | (static_cast<uint32_t>(float_to_bf16_bits(hi)) << 16);
}
// Elements past the row's end are 0.
template <bool VEC, int E>
__device__ __forceinline__ void load_row(const uint16_t* row, int d, float (&v)[E]) {
    if constexpr (VEC) {
        uint4 w[E / 8];
#pragma unroll
        for (int k = 0; k < E / 8; ++k)
            w[k] = col_of<true>(8 * k) < d ? *reinterpret_cast<const uint4*>(row + col_of<true>(8 * k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < E / 8; ++k) unpack8(w[k], v + 8 * k);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = col_of<false>(e) < d ? bf16_bits_to_float(row[col_of<false>(e)]) : 0.f;
    }
}
template <bool VEC, int E>
__device__ __forceinline__ void load_row(const float* row, int d, float (&v)[E]) {
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < E / 4; ++k) {
            const int c = col_of<true>(4 * k);
            const float4 w = c < d ? *reinterpret_cast<const float4*>(row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[4 * k] = w.x;
            v[4 * k + 1] = w.y;
            v[4 * k + 2] = w.z;
            v[4 * k + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = col_of<false>(e) < d ? row[col_of<false>(e)] : 0.f;
    }
}
template <bool VEC, int E>
__device__ __forceinline__ void store_row(uint16_t* row, int d, const float (&v)[E]) {
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < E / 8; ++k) {
            const float* f = v + 8 * k;
            if (col_of<true>(8 * k) < d)
                *reinterpret_cast<uint4*>(row + col_of<true>(8 * k)) =
                    make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col_of<false>(e) < d) row[col_of<false>(e)] = float_to_bf16_bits(v[e]);
    }
}
template <bool VEC, int E>
__device__ __forceinline__ void store_row(float* row, int d, const float (&v)[E]) {
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < E / 4; ++k)
            if (col_of<true>(4 * k) < d)
                *reinterpret_cast<float4*>(row + col_of<true>(4 * k)) =
                    make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col_of<false>(e) < d) row[col_of<false>(e)] = v[e];
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

// One block per row, which stays in registers: every element is read once and written once.
// Bound by HBM; 32 elements a thread keep 100 KB and more of loads in flight per multiprocessor.
template <bool VEC, int E, bool F32>
__global__ void __launch_bounds__(1024 * 8 / (E > 8 ? E : 8)) block_norm_rows_kernel(const NormFwdArgs a) {
    using H = std::conditional_t<F32, float, uint16_t>;
    __shared__ float red[2][32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t m = blockIdx.x, base = m * a.d;
    const int d = static_cast<int>(a.d);
    float h[E];
    load_row<VEC, E>(static_cast<const H*>(a.h) + base, d, h);
    if (a.y) {
        float y[E], f[E];
        load_row<VEC, E>(a.y + base, d, y);
        if (a.post) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(y[e], y[e], s);
            const float rp = rsqrtf(block_sum1(s, red[0]) / static_cast<float>(d) + a.eps);
            if (a.w_post) load_row<VEC, E>(a.w_post, d, f);
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] *= a.w_post ? rp * (a.w_offset + f[e]) : rp;
        }
        if (a.gate) {
            load_row<VEC, E>(a.gate + m * a.ld_gate, d, f);
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] *= f[e];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = fmaf(a.alpha, h[e], y[e]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] *= a.alpha;
    }
    if (a.h_out) store_row<VEC, E>(static_cast<H*>(a.h_out) + base, d, h);
    if (a.x) {
        float s = 0.f, f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(h[e], h[e], s);
        if (a.w_pre) load_row<VEC, E>(a.w_pre, d, f);
        const float r = rsqrtf(block_sum1(s, red[1]) / static_cast<float>(d) + a.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] *= a.w_pre ? r * (a.w_offset + f[e]) : r;
        store_row<VEC, E>(a.x + base, d, h);
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

// Blocks take rows in turn; block b keeps its sums over rows for the vectors' gradients in
// part[k][b][d] (k = g_w_pre, g_w_post, g_gate), each column always by the same thread.
__global__ void __launch_bounds__(kNormThreads) block_norm_grad_any_kernel(const NormBwdArgs a) {
    __shared__ float red[96];
    pdl_wait();
    pdl_launch_dependents();
    const float inv_d = 1.0f / static_cast<float>(a.d);
    const bool row_gate = a.gate && a.ld_gate > 0;
    float* part[3];
    for (int k = 0; k < 3; ++k)
        part[k] = a.part[k] ? a.part[k] + static_cast<int64_t>(blockIdx.x) * a.d : nullptr;
    for (int k = 0; k < 3; ++k)
        if (part[k])
            for (int64_t i = threadIdx.x; i < a.d; i += kNormThreads) part[k][i] = 0.f;
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
        const float rp = rsqrtf(s[2] * inv_d + a.eps);
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
            if (part[0] && a.gx) part[0][i] += bf16_bits_to_float(a.gx[base + i]) * hn;
            if (a.y) {
                const float gt = gate ? bf16_bits_to_float(gate[i]) : 1.f;
                const float y = bf16_bits_to_float(a.y[base + i]);
                const float w = ld_w(a.w_post, i, a.w_offset);
                const float yn = y * rp, z = a.post ? yn * w : y, dz = dh * gt;
                if (part[1]) part[1][i] += dz * yn;
                if (part[2]) part[2][i] += dh * z;
                if (row_gate && a.g_gate_rows) a.g_gate_rows[base + i] = float_to_bf16_bits(dh * z);
                if (a.gy) a.gy[base + i] = float_to_bf16_bits(a.post ? rp * (w * dz - yn * cp) : dz);
            }
            if (a.gh) st_h(a.gh, base + i, a.h_f32, a.alpha * dh);
        }
    }
}

// ------------------------------------------------------------------ backward, rows in shared memory
//
// The vectors' gradients are sums over the rows, so a block takes rows in turn and its threads keep
// their columns' sums in registers (kGradE columns a thread).  Rows come in by bulk copies, a ring
// ahead of the arithmetic.  All that a row's gradients need of the whole row are six sums: with
// v = w_pre gx, r = 1 / q(h'), rp = 1 / q(y) and b = w_post gate y,
//   sum h'^2, sum v h', sum y^2, sum b gh', sum b v, sum b h'
// give c = mean(v h'^) / q(h') and, as dh' = gh' + r v - r h' c, also
//   sum w_post dz y = sum b gh' + r sum b v - r c sum b h',
// so that one block-wide reduction a row is enough.
constexpr int kGradE = 16;

struct NormBwdSmem {
    int stages;
    uint32_t stage_bytes;
    uint32_t off_gx, off_h, off_gh, off_gate;  // in a stage; y is first
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

template <bool VEC, bool F32>
__global__ void __launch_bounds__(512, 1) block_norm_grad_rows_kernel(const NormBwdArgs a, const NormBwdSmem sm) {
    using H = std::conditional_t<F32, float, uint16_t>;
    constexpr int E = kGradE;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][6][16];
    __shared__ __align__(8) uint64_t bar[4];
    const int d = static_cast<int>(a.d), warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const uint32_t bar0 = tc::smem_u32(bar);
    if (threadIdx.x == 0) {
        for (int s = 0; s < sm.stages; ++s) tc::mbar_init(bar0 + 8u * s, 1);
        tc::mbar_fence_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const bool row_gate = a.gate && a.ld_gate > 0;
    const uint16_t* src16[3] = {a.y, a.gx, row_gate ? a.gate : nullptr};
    const uint32_t off16[3] = {0u, sm.off_gx, sm.off_gate};
    const void* srch[2] = {a.h_out, a.gh_out};
    const uint32_t offh[2] = {sm.off_h, sm.off_gh};
    const int64_t total16 = a.M * a.d * 2, totalh = a.M * a.d * static_cast<int64_t>(sizeof(H));

    auto load = [&](int64_t m, int s) {  // one thread
        const int64_t f16 = m * a.d * 2, fh = m * a.d * static_cast<int64_t>(sizeof(H));
        bool odd16, oddh;
        const uint32_t n16 = span_bytes(f16, d * 2u, total16, odd16), nh = span_bytes(fh, d * sizeof(H), totalh, oddh);
        uint8_t* st = smem + s * sm.stage_bytes;
        uint32_t tx = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) tx += src16[i] ? n16 : 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) tx += srch[i] ? nh : 0u;
        if (odd16) {  // next to the tensor's end only
            for (int i = 0; i < 3; ++i)
                if (src16[i])
                    for (int64_t b = std::max((f16 + d * 2) & ~int64_t{15}, f16); b < f16 + d * 2; b += 2)
                        *reinterpret_cast<uint16_t*>(st + off16[i] + (b - (f16 & ~int64_t{15}))) = src16[i][b / 2];
        }
        if (oddh) {
            for (int i = 0; i < 2; ++i)
                if (srch[i])
                    for (int64_t b = std::max((fh + d * static_cast<int64_t>(sizeof(H))) & ~int64_t{15}, fh);
                         b < fh + d * static_cast<int64_t>(sizeof(H)); b += sizeof(H))
                        *reinterpret_cast<H*>(st + offh[i] + (b - (fh & ~int64_t{15}))) =
                            static_cast<const H*>(srch[i])[b / static_cast<int64_t>(sizeof(H))];
        }
        tc::mbar_arrive_expect_tx(bar0 + 8u * s, tx);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (src16[i] && n16)
                tc::bulk_load(tc::smem_u32(st + off16[i]),
                              reinterpret_cast<const uint8_t*>(src16[i]) + (f16 & ~int64_t{15}), n16, bar0 + 8u * s);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (srch[i] && nh)
                tc::bulk_load(tc::smem_u32(st + offh[i]), static_cast<const uint8_t*>(srch[i]) + (fh & ~int64_t{15}), nh,
                              bar0 + 8u * s);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < sm.stages; ++s)
            if (blockIdx.x + static_cast<int64_t>(s) * gridDim.x < a.M) load(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);

    // the vectors, two bf16 to a register
    uint32_t wpre[E / 2], wpost[E / 2], gt[E / 2];
    auto load_vector = [&](const uint16_t* w, uint32_t (&out)[E / 2]) {
        float f[E];
        if (w) load_row<VEC, E>(w, d, f);
#pragma unroll
        for (int e = 0; e < E; e += 2)  // bf16 values: exact
            out[e / 2] = w ? (__float_as_uint(f[e]) >> 16) | (__float_as_uint(f[e + 1]) & 0xFFFF0000u) : 0x3F803F80u;
    };
    load_vector(a.w_pre, wpre);
    load_vector(a.post ? a.w_post : nullptr, wpost);
    load_vector(row_gate ? nullptr : a.gate, gt);
    const float off_pre = a.w_pre ? a.w_offset : 0.f, off_post = a.post && a.w_post ? a.w_offset : 0.f;
    auto half = [](const uint32_t (&w)[E / 2], int e) {
        return __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    };
    float acc[3][E];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[k][e] = 0.f;
    const float inv_d = 1.0f / static_cast<float>(d);

    uint32_t it = 0;
    int s = 0;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, ++it) {
        // a wait that gives up leaves stale rows behind; the error word tells
        tc::mbar_wait(bar0 + 8u * s, (it / sm.stages) & 1u, a.err);
        const uint8_t* st = smem + s * sm.stage_bytes;
        const int64_t base = m * a.d;
        const uint32_t lead16 = static_cast<uint32_t>(base * 2) & 15u;
        const uint32_t leadh = static_cast<uint32_t>(base * static_cast<int64_t>(sizeof(H))) & 15u;
        // 8 elements from a piece's first e (VEC) or one (else)
        constexpr int P = VEC ? 8 : 1;
        auto get16 = [&](uint32_t off, bool there, int e, float (&v)[P]) {
            const int c = col_of<VEC>(e);
            const bool in = there && c < d;
            const uint16_t* p = reinterpret_cast<const uint16_t*>(st + off + (VEC ? 0u : lead16)) + c;
            if constexpr (VEC)
                unpack8(in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0), v);
            else
                v[0] = in ? bf16_bits_to_float(*p) : 0.f;
        };
        auto geth = [&](uint32_t off, bool there, int e, float (&v)[P]) {
            const int c = col_of<VEC>(e);
            const bool in = there && c < d;
            const H* p = reinterpret_cast<const H*>(st + off + (VEC ? 0u : leadh)) + c;
            if constexpr (VEC && F32) {
                const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 f0 = in ? reinterpret_cast<const float4*>(p)[0] : z, f1 = in ? reinterpret_cast<const float4*>(p)[1] : z;
                v[0] = f0.x, v[1] = f0.y, v[2] = f0.z, v[3] = f0.w, v[4] = f1.x, v[5] = f1.y, v[6] = f1.z, v[7] = f1.w;
            } else if constexpr (VEC) {
                unpack8(in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0), v);
            } else if constexpr (F32) {
                v[0] = in ? *p : 0.f;
            } else {
                v[0] = in ? bf16_bits_to_float(*p) : 0.f;
            }
        };
        float sum[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e0 = 0; e0 < E; e0 += P) {
            float y[P], gx[P], h[P], gh[P], gr[P];
            get16(0u, a.y != nullptr, e0, y);
            get16(sm.off_gx, a.gx != nullptr, e0, gx);
            geth(sm.off_h, true, e0, h);
            geth(sm.off_gh, a.gh_out != nullptr, e0, gh);
            if (row_gate) get16(sm.off_gate, true, e0, gr);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float v = (off_pre + half(wpre, e0 + i)) * gx[i];
                const float b = (off_post + half(wpost, e0 + i)) * (row_gate ? gr[i] : half(gt, e0 + i)) * y[i];
                sum[0] = fmaf(h[i], h[i], sum[0]);
                sum[1] = fmaf(v, h[i], sum[1]);
                sum[2] = fmaf(y[i], y[i], sum[2]);
                sum[3] = fmaf(b, gh[i], sum[3]);
                sum[4] = fmaf(b, v, sum[4]);
                sum[5] = fmaf(b, h[i], sum[5]);
            }
        }
#pragma unroll
        for (int k = 0; k < 6; ++k) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum[k] += __shfl_xor_sync(0xFFFFFFFFu, sum[k], o);
            if (lane == 0) red[it & 1][k][warp] = sum[k];
        }
        __syncthreads();  // and every thread is done with the last row
        if (threadIdx.x == 0 && it > 0) {
            const int64_t ahead = m + static_cast<int64_t>(sm.stages - 1) * gridDim.x;
            const int ps = s == 0 ? sm.stages - 1 : s - 1;
            if (ahead < a.M) {
                tc::fence_proxy_async_smem();
                load(ahead, ps);
            }
        }
#pragma unroll
        for (int k = 0; k < 6; ++k) {
            sum[k] = 0.f;
            for (int w = 0; w < nw; ++w) sum[k] += red[it & 1][k][w];
        }
        const float r = rsqrtf(sum[0] * inv_d + a.eps);
        const float c = sum[1] * inv_d * r * r;  // mean(v h'^) / q(h')
        const float rp = a.post ? rsqrtf(sum[2] * inv_d + a.eps) : 1.f;
        const float cp = (sum[3] + r * sum[4] - r * c * sum[5]) * inv_d * rp;  // mean(w_post dz y^)
#pragma unroll
        for (int e0 = 0; e0 < E; e0 += P) {
            float y[P], gx[P], h[P], gh[P], gr[P], gy[P], gg[P];
            get16(0u, a.y != nullptr, e0, y);
            get16(sm.off_gx, a.gx != nullptr, e0, gx);
            geth(sm.off_h, true, e0, h);
            geth(sm.off_gh, a.gh_out != nullptr, e0, gh);
            if (row_gate) get16(sm.off_gate, true, e0, gr);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float hn = h[i] * r, gate = row_gate ? gr[i] : half(gt, e0 + i);
                const float w = off_post + half(wpost, e0 + i);
                const float dh = gh[i] + r * ((off_pre + half(wpre, e0 + i)) * gx[i]) - hn * c;
                acc[0][e0 + i] = fmaf(gx[i], hn, acc[0][e0 + i]);
                const float yn = y[i] * rp, dz = dh * gate, z = yn * w;
                acc[1][e0 + i] = fmaf(dz, yn, acc[1][e0 + i]);
                gg[i] = dh * z;
                acc[2][e0 + i] += gg[i];
                gy[i] = a.post ? rp * (w * dz - yn * cp) : dz;
                gh[i] = a.alpha * dh;
            }
            const int col = col_of<VEC>(e0);
            if (col < d) {
                if constexpr (VEC) {
                    auto pack = [](const float (&f)[P]) {
                        return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
                    };
                    if (a.gy) *reinterpret_cast<uint4*>(a.gy + base + col) = pack(gy);
                    if (row_gate && a.g_gate_rows) *reinterpret_cast<uint4*>(a.g_gate_rows + base + col) = pack(gg);
                    if constexpr (F32) {
                        if (a.gh) {
                            float4* to = reinterpret_cast<float4*>(static_cast<float*>(a.gh) + base + col);
                            to[0] = make_float4(gh[0], gh[1], gh[2], gh[3]);
                            to[1] = make_float4(gh[4], gh[5], gh[6], gh[7]);
                        }
                    } else if (a.gh) {
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.gh) + base + col) = pack(gh);
                    }
                } else {
                    if (a.gy) a.gy[base + col] = float_to_bf16_bits(gy[0]);
                    if (row_gate && a.g_gate_rows) a.g_gate_rows[base + col] = float_to_bf16_bits(gg[0]);
                    if (a.gh) st_h(a.gh, base + col, F32, gh[0]);
                }
            }
        }
        if (++s == sm.stages) s = 0;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (a.part[k]) store_row<VEC, E>(a.part[k] + static_cast<int64_t>(blockIdx.x) * a.d, d, acc[k]);
}

// out[k][i] = sum over the blocks' partial sums, in fp64: 8 threads a column, each with every eighth
// block, then the 8 in order.
__global__ void __launch_bounds__(256) norm_vector_sums_kernel(const NormSumArgs a) {
    __shared__ double part[8][32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
    const int k = blockIdx.y, g = threadIdx.x >> 5;
    if (!a.out[k]) return;
    double s = 0.0;
    if (i < a.d) {
#pragma unroll 8
        for (int b = g; b < a.blocks; b += 8) s += static_cast<double>(a.part[k][static_cast<int64_t>(b) * a.d + i]);
    }
    part[g][threadIdx.x & 31] = s;
    __syncthreads();
    if (g == 0 && i < a.d) {
        for (int j = 1; j < 8; ++j) s += part[j][threadIdx.x];
        a.out[k][i] = static_cast<float>(s);
    }
}

}  // namespace nq

namespace {

constexpr size_t kNormSmemMax = 226 * 1024;

// Threads for a row of d channels at E elements each.
int row_threads(int64_t d, int E) { return static_cast<int>((d + 32 * E - 1) / (32 * E) * 32); }

// Backward: blocks that share the rows.  Rows of up to 8192 channels take 512 threads a
// multiprocessor with 128 registers each (16 columns' sums); wider ones two blocks of any size.
int grad_blocks(int64_t d, int64_t M) {
    const int per_sm = d <= 512 * nq::kGradE ? std::max(1, std::min(16, 512 / row_threads(d, nq::kGradE))) : 2;
    return static_cast<int>(std::min<int64_t>(M, static_cast<int64_t>(per_sm) * nq_host::sm_count()));
}

template <bool VEC, bool F32>
const void* rows_kernel(int E) {
    return E == 8    ? reinterpret_cast<const void*>(nq::block_norm_rows_kernel<VEC, 8, F32>)
           : E == 16 ? reinterpret_cast<const void*>(nq::block_norm_rows_kernel<VEC, 16, F32>)
                     : reinterpret_cast<const void*>(nq::block_norm_rows_kernel<VEC, 32, F32>);
}

}  // namespace

nq_status nq_launch_block_norm(const nq::NormFwdArgs& a, int64_t M, cudaStream_t stream, bool pdl) {
    nq::NormFwdArgs args = a;
    void* kargs[] = {&args};
    // Few rows: as many threads a row as there are pieces of 8, for the latency; many: 32 elements a
    // thread, for loads in flight at few threads.  A block has at most 8192 / E threads of E
    // elements, so that its registers fit: rows over 8192 channels go through the other kernel.
    int E = 8;
    const bool vec = a.d % 8 == 0 && a.ld_gate % 8 == 0;
    if (M >= 4 * static_cast<int64_t>(nq_host::sm_count())) E = vec ? 32 : 16;
    const void* fn = reinterpret_cast<const void*>(nq::block_norm_any_kernel);
    int threads = nq::kNormThreads;
    if (a.d <= 8192) {
        fn = vec ? (a.h_f32 ? rows_kernel<true, true>(E) : rows_kernel<true, false>(E))
                 : (a.h_f32 ? rows_kernel<false, true>(E) : rows_kernel<false, false>(E));
        threads = row_threads(a.d, E);
    }
    return nq_host::launch_pdl(fn, dim3(static_cast<unsigned>(M)), dim3(threads), 0, stream, kargs, pdl) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}

size_t nq_block_norm_grad_ws(int64_t d, int64_t M) {
    return NQ_WS_HEADER_BYTES + 3 * static_cast<size_t>(grad_blocks(d, M)) * d * sizeof(float);
}

nq_status nq_launch_block_norm_grad(const nq::NormBwdArgs& a, float* g_w_pre, float* g_w_post, float* g_gate, void* ws,
                                    cudaStream_t stream, bool pdl) {
    const int blocks = grad_blocks(a.d, a.M);
    nq::NormBwdArgs args = a;
    args.err = nq_host::error_word();
    nq::NormSumArgs sum{};
    float* out[3] = {g_w_pre, g_w_post, g_gate};
    float* p = reinterpret_cast<float*>(static_cast<char*>(ws) + NQ_WS_HEADER_BYTES);
    bool any = false;
    for (int k = 0; k < 3; ++k) {
        args.part[k] = out[k] ? p + static_cast<int64_t>(k) * blocks * a.d : nullptr;
        sum.part[k] = args.part[k];
        sum.out[k] = out[k];
        any = any || out[k];
    }
    sum.d = a.d;
    sum.blocks = blocks;
    const bool row_gate = a.gate && a.ld_gate > 0;
    bool launched = false;
    if (a.d <= 512 * nq::kGradE && !(row_gate && a.ld_gate != a.d)) {
        // rows in shared memory; a row that does not start on 16 bytes brings up to 15 more before and after
        nq::NormBwdSmem sm{};
        auto region = [&](bool there, size_t elem) {
            return there ? static_cast<uint32_t>((a.d * elem + 30 + 127) / 128 * 128) : 0u;
        };
        const size_t he = a.h_f32 ? 4 : 2;
        sm.off_gx = region(a.y != nullptr, 2);
        sm.off_h = sm.off_gx + region(a.gx != nullptr, 2);
        sm.off_gh = sm.off_h + region(true, he);
        sm.off_gate = sm.off_gh + region(a.gh_out != nullptr, he);
        sm.stage_bytes = sm.off_gate + region(row_gate, 2);
        const int threads = row_threads(a.d, nq::kGradE);
        const size_t share = kNormSmemMax / std::max(1, std::min(16, 512 / threads)) - 2048;
        sm.stages = static_cast<int>(std::max<size_t>(2, std::min<size_t>(4, share / sm.stage_bytes)));
        if (static_cast<size_t>(sm.stages) * sm.stage_bytes <= kNormSmemMax) {
            const bool vec = a.d % 8 == 0;
            const void* fns[4] = {reinterpret_cast<const void*>(nq::block_norm_grad_rows_kernel<false, false>),
                                  reinterpret_cast<const void*>(nq::block_norm_grad_rows_kernel<false, true>),
                                  reinterpret_cast<const void*>(nq::block_norm_grad_rows_kernel<true, false>),
                                  reinterpret_cast<const void*>(nq::block_norm_grad_rows_kernel<true, true>)};
            static std::atomic<bool> attr_done[64];  // per device; setting an attribute twice is harmless
            int dev = 0;
            cudaGetDevice(&dev);
            if (dev < 0 || dev >= 64) return NQ_ERR_DEVICE;
            if (!attr_done[dev].load(std::memory_order_acquire)) {
                for (const void* f : fns)
                    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kNormSmemMax)) != cudaSuccess)
                        return NQ_ERR_LAUNCH;
                attr_done[dev].store(true, std::memory_order_release);
            }
            void* kargs[] = {&args, &sm};
            if (nq_host::launch_pdl(fns[(vec ? 2 : 0) + (a.h_f32 ? 1 : 0)], dim3(blocks), dim3(threads),
                                    static_cast<size_t>(sm.stages) * sm.stage_bytes, stream, kargs, pdl) != cudaSuccess)
                return NQ_ERR_LAUNCH;
            launched = true;
        }
    }
    if (!launched) {
        void* kargs[] = {&args};
        if (nq_host::launch_pdl(reinterpret_cast<const void*>(nq::block_norm_grad_any_kernel), dim3(blocks),
                                dim3(nq::kNormThreads), 0, stream, kargs, pdl) != cudaSuccess)
            return NQ_ERR_LAUNCH;
    }
    if (!any) return NQ_OK;
    void* sargs[] = {&sum};
    return nq_host::launch_pdl(reinterpret_cast<const void*>(nq::norm_vector_sums_kernel),
                               dim3(static_cast<unsigned>((a.d + 31) / 32), 3), dim3(256), 0, stream, sargs,
                               pdl) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}
