// norm.cuh -- arguments of the block-norm kernels (norm.cu), filled by the C ABI (api.cu).
#pragma once

#include <stdint.h>

#include "nq.h"

namespace nq {

struct NormFwdArgs {
    const uint16_t* y;      // [M][d] bf16 or nullptr (no block output)
    const void* h;          // [M][d] residual
    void* h_out;            // [M][d] or nullptr
    uint16_t* x;            // [M][d] bf16 or nullptr
    const uint16_t* gate;   // bf16, row m at gate + m ld_gate (ld_gate 0: shared) or nullptr (ones)
    const uint16_t* w_post; // [d] bf16 or nullptr (ones)
    const uint16_t* w_pre;
    int64_t d, ld_gate;
    float alpha, eps, w_offset;
    bool post, h_f32;
    unsigned int* err;
};

struct NormBwdArgs {
    const uint16_t* y;
    const void* h_out;
    const uint16_t* gx;     // [M][d] bf16 or nullptr (zero)
    const void* gh_out;     // [M][d] or nullptr (zero)
    const uint16_t* gate;
    const uint16_t* w_post;
    const uint16_t* w_pre;
    void* gh;               // outputs, each may be nullptr
    uint16_t* gy;
    uint16_t* g_gate_rows;  // [M][d] bf16, for a gate per row
    // [blocks][part_ld] sums over a block's rows, or nullptr: gx h'^, and dh' y^ (times a gate per row)
    float* part[2];
    int64_t part_ld;
    int64_t M, d, ld_gate;
    float alpha, eps, w_offset;
    bool post, h_f32;
    unsigned int* err;
};

struct NormSumArgs {
    const float* part[2];
    int64_t part_ld, d;
    int blocks;
    const uint16_t* gate;    // shared gate or nullptr (ones): g_w_post = gate sum dh' y^
    const uint16_t* w_post;  // nullptr (ones): g_gate = (w_offset + w_post) sum dh' y^
    float w_offset;
    float *g_w_pre, *g_w_post, *g_gate;  // each may be nullptr
};

}  // namespace nq

nq_status nq_launch_block_norm(const nq::NormFwdArgs& a, int64_t M, cudaStream_t stream, bool pdl);
size_t nq_block_norm_grad_ws(int64_t d, int64_t M);
nq_status nq_launch_block_norm_grad(const nq::NormBwdArgs& a, float* g_w_pre, float* g_w_post, float* g_gate, void* ws,
                                    cudaStream_t stream, bool pdl);
