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
#include "nq_common.cuh"
#include "norm.cuh"

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

// out[k][i] = sum over the blocks' partial sums, in fp64, in order.
__global__ void __launch_bounds__(256) norm_vector_sums_kernel(const NormSumArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int k = blockIdx.y;
    if (i >= a.d || !a.out[k]) return;
    double s = 0.0;
    for (int b = 0; b < a.blocks; ++b) s += static_cast<double>(a.part[k][static_cast<int64_t>(b) * a.d + i]);
    a.out[k][i] = static_cast<float>(s);
}

}  // namespace nq

namespace {
// Blocks that share the rows of a backward pass: two per multiprocessor.
int grad_blocks(int64_t M) {
    const int64_t cap = 2 * static_cast<int64_t>(nq_host::sm_count());
    return static_cast<int>(M < cap ? M : cap);
}
}  // namespace

nq_status nq_launch_block_norm(const nq::NormFwdArgs& a, int64_t M, cudaStream_t stream, bool pdl) {
    nq::NormFwdArgs args = a;
    void* kargs[] = {&args};
    return nq_host::launch_pdl(reinterpret_cast<const void*>(nq::block_norm_any_kernel),
                               dim3(static_cast<unsigned>(M)), dim3(nq::kNormThreads), 0, stream, kargs,
                               pdl) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}

size_t nq_block_norm_grad_ws(int64_t d, int64_t M) {
    return NQ_WS_HEADER_BYTES + 3 * static_cast<size_t>(grad_blocks(M)) * d * sizeof(float);
}

nq_status nq_launch_block_norm_grad(const nq::NormBwdArgs& a, float* g_w_pre, float* g_w_post, float* g_gate, void* ws,
                                    cudaStream_t stream, bool pdl) {
    const int blocks = grad_blocks(a.M);
    nq::NormBwdArgs args = a;
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
    void* kargs[] = {&args};
    if (nq_host::launch_pdl(reinterpret_cast<const void*>(nq::block_norm_grad_any_kernel), dim3(blocks),
                            dim3(nq::kNormThreads), 0, stream, kargs, pdl) != cudaSuccess)
        return NQ_ERR_LAUNCH;
    if (!any) return NQ_OK;
    void* sargs[] = {&sum};
    return nq_host::launch_pdl(reinterpret_cast<const void*>(nq::norm_vector_sums_kernel),
                               dim3(static_cast<unsigned>((a.d + 255) / 256), 3), dim3(256), 0, stream, sargs,
                               pdl) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_LAUNCH;
}
