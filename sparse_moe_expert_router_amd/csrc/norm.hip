// Residual addition with root-mean-square norm, and its gradients.
//
// Forward, per row of H values:
//   s = round_res(x + residual)      (the residual as it is stored; s = x without one)
//   r = 1 / sqrt(mean(s^2) + eps)
//   v = (s r) (offset + w)           -> y = bf16(v), or E4M3 codes of v with one scale per 128 values (fp8.h)
// Backward, with h = s r and u = dy (offset + w):
//   dx = r (u - h mean(u h)) + dres,   dw = sum over rows of dy h
//
// Both are bound by memory: every value is read once and held in registers
// between the sum over its row and its use.  A thread holds C pieces of 8
// neighbouring values (16 or 32 bytes), piece c of thread t being values
// 8 (c n + t) .. +7 of the row for n threads, so a group of 128 values lies in
// 16 neighbouring lanes.  A workgroup of as few waves as the row needs takes
// one row after another.
#include "fp8.h"
#include "kernels.h"
#include "rows.h"

namespace moe {

constexpr int kMaxWaves = 16;

// Sum over the workgroup; `red` holds one slot of partial sums, alternated by
// the caller from call to call so that one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int waves) {
    v = wave_sum_f32(v);
    if (waves == 1) return v;
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < waves; ++i) t += red[i];
    return t;
}

// Maximum over the 16 lanes of a row of lanes, in every lane of it.
__device__ __forceinline__ uint32_t max16_u32(uint32_t v) {
    v = max8_u32(v);
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));  // row_mirror
}

template <int C>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
    __shared__ float red[2][kMaxWaves];
    const int n = blockDim.x, waves = n / kWave, t = threadIdx.x;
    const int nb = fp8_blocks(a.H);
    bool in[C];
    f32x8_t gain[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = 8 * (c * n + t);
        in[c] = i < a.H;
        gain[c] = in[c] ? load8(a.w, i, a.w_f32) + a.offset : f32x8_t(0.0f);
    }
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, flip ^= 1) {
        f32x8_t s[C];
        float sq = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (c * n + t);
            s[c] = f32x8_t(0.0f);
            if (in[c]) {
                s[c] = load8(a.x, row * a.ldx + i, a.x_f32);
                if (a.res) {
                    s[c] += load8(a.res, row * a.ldr + i, a.r_f32);
                    if (!a.r_f32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) s[c][j] = bf16_to_f32(f32_to_bf16_bits(s[c][j]));
                    }
                    store8(a.res_out, row * a.ldro + i, a.r_f32, s[c]);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fmaf(s[c][j], s[c][j], sq);
        }
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(row_sum(sq, red[flip], waves), (float)a.H) + a.eps));
        if (a.rstd && t == 0) a.rstd[row] = r;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (c * n + t);
            const f32x8_t v = s[c] * r * gain[c];
            if (a.y && in[c]) store8(a.y, row * a.ldy + i, 0, v);
            if (a.codes) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
                const float sc = fp8_scale(max16_u32(m));
                const Fp8Div d = fp8_div(in[c] ? sc : 1.0f);
                if (in[c]) {
                    const uint2 q = make_uint2(fp8_pack4(v[0], v[1], v[2], v[3], d), fp8_pack4(v[4], v[5], v[6], v[7], d));
                    *reinterpret_cast<uint2*>(a.codes + row * a.H + i) = q;
                    if (t % 16 == 0) a.scales[row * nb + i / kFp8Block] = sc;
                }
            }
        }
    }
}

template <int C>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormBwdArgs a, float* __restrict__ part) {
    __shared__ float red[2][kMaxWaves];
    const int n = blockDim.x, waves = n / kWave, t = threadIdx.x;
    bool in[C];
    f32x8_t gain[C], dw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = 8 * (c * n + t);
        in[c] = i < a.H;
        gain[c] = in[c] ? load8(a.w, i, a.w_f32) + a.offset : f32x8_t(0.0f);
        dw[c] = f32x8_t(0.0f);
    }
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, flip ^= 1) {
        const float r = a.rstd[row];
        f32x8_t h[C], u[C];
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (c * n + t);
            h[c] = u[c] = f32x8_t(0.0f);
            if (in[c]) {
                h[c] = load8(a.s, row * a.lds + i, a.s_f32) * r;
                const f32x8_t dy = load8(a.dy, row * a.ldy + i, a.y_f32);
                dw[c] += dy * h[c];
                u[c] = dy * gain[c];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) dot = fmaf(u[c][j], h[c][j], dot);
        }
        const float mean = __fdiv_rn(row_sum(dot, red[flip], waves), (float)a.H);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (c * n + t);
            if (!in[c]) continue;
            f32x8_t d = (u[c] - h[c] * mean) * r;
            if (a.dres) d += load8(a.dres, row * a.lddr + i, a.s_f32);
            store8(a.dx, row * a.lddx + i, a.s_f32, d);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = 8 * (c * n + t);
        if (in[c]) store8(part, (int64_t)blockIdx.x * a.H + i, 1, dw[c]);
    }
}

// dw [H] = sum of the `parts` partial rows, in a fixed order: 64 columns a
// workgroup, its 16 waves each every sixteenth row, then the waves in turn.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ part, int parts, int H, float* __restrict__ dw) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
    const int col = blockIdx.x * 64 + lane;
    float v = 0.0f;
    if (col < H)
        for (int p = w; p < parts; p += 16) v += part[(size_t)p * H + col];
    red[w][lane] = v;
    __syncthreads();
    if (w == 0 && col < H) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += red[i][lane];
        dw[col] = s;
    }
}

namespace {

// Pieces a thread for a row of H values: one while 16 waves hold the row so, else two (kNormMaxH values).
int pieces(int H) { return H <= 8 * 64 * kMaxWaves ? 1 : 2; }
int waves_for(int H, int c) { return (H + 512 * c - 1) / (512 * c); }

// Workgroups: each compute unit holds 32 waves at most, two rounds of them.
int norm_grid(int T, int waves) {
    const int most = 256 * (32 / waves) * 2;
    return T < most ? T : most;
}
int bwd_grid(int T, int H) {
    const int most = 256 * (16 / waves_for(H, pieces(H)) + 1);
    return T < most ? T : most;
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s) {
    const int c = pieces(a.H), w = waves_for(a.H, c);
    const dim3 grid(norm_grid(a.T, w)), block(64 * w);
    if (c == 1) hipLaunchKernelGGL((norm_kernel<1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((norm_kernel<2>), grid, block, 0, s, a);
    return hipGetLastError();
}

size_t norm_bwd_ws_bytes(int T, int H) { return (size_t)bwd_grid(T, H) * H * sizeof(float); }

hipError_t launch_add_rmsnorm_backward(const NormBwdArgs& a, void* ws, hipStream_t s) {
    const int c = pieces(a.H), w = waves_for(a.H, c);
    const int parts = a.T ? bwd_grid(a.T, a.H) : 0;
    float* part = static_cast<float*>(ws);
    if (parts) {
        const dim3 grid(parts), block(64 * w);
        if (c == 1) hipLaunchKernelGGL((norm_bwd_kernel<1>), grid, block, 0, s, a, part);
        else hipLaunchKernelGGL((norm_bwd_kernel<2>), grid, block, 0, s, a, part);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(norm_dw_kernel, dim3((a.H + 63) / 64), dim3(1024), 0, s, part, parts, a.H, a.dw);
    return hipGetLastError();
}

}  // namespace moe
