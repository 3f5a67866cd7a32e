// The dense W8A8 product for few rows: E4M3 codes on both sides, fp32 scales per
// 128 inputs (rows) and per 128 x 128 block (weights), gfx950's 16 x 16 x 128 FP8
// MFMA (fp32 outputs: the bf16 MFMA on widened codes, see mfma_fp8).  One call of
// it covers one block of 128 inputs of 16 outputs x 16 rows; its result is
// multiplied by the two scales and added to an fp32 accumulator:
//   y[m][n] += (sa[m][kb] * sw[n / 128][kb]) * sum_i a[m][i] w[n][i].
// The weights are the MFMA's row operand, so a lane ends up with four
// neighbouring outputs of one row.
//
// With few rows the weights' bytes and the waits for them bound the call.  They
// go from memory straight into registers, each byte once per row tile; rows are
// read from the caches.  A workgroup has only 16 outputs and splits the inputs
// over its 8 waves, which are joined through LDS in a fixed order: enough
// workgroups for the chip, and a wait of a few blocks for each.  (1 x 2560 x
// 2560: 8.3 us, 7 of them the call itself; 1 x 16384 x 8192: 26 us, 5.2 TB/s.)
#include "fp8.h"
#include "ffn_internal.h"
#include "fp8_internal.h"

namespace moe {

// One wave's product of 16 weight rows with TF groups of 16 activation rows over
// blocks kb0, kb0 + kstep, ... < KB of 128 inputs.  wr / ar: buffers whose rows
// past the end read as zero; woff / aoff: the lane's byte offset of its row;
// kend: bytes of a row (a multiple of 16).
template <int TF, bool kExact>
__device__ __forceinline__ void fp8_wave_product(f32x4_t (&acc)[TF], __amdgpu_buffer_rsrc_t wr, uint32_t woff,
                                                 __amdgpu_buffer_rsrc_t ar, const uint32_t (&aoff)[TF],
                                                 __amdgpu_buffer_rsrc_t sr, const uint32_t (&soff)[TF], const float* sw,
                                                 int kb0, int kstep, int KB, int kend, int g) {
    constexpr int U = TF == 1 ? 5 : 4;  // blocks loaded before the first is used
    for (int kbase = kb0; kbase < KB; kbase += U * kstep) {
        i32x8_t w[U], a[U][TF];
        float s[U][TF];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // a lane group's 32 inputs: pieces g and g + 4 of the block's
            // eight.  Past the row's end both sides and the scales read zero.
            const int kb = kbase + u * kstep;
            const uint32_t k0 = (uint32_t)kb * 128u + 16u * (uint32_t)g, k1 = k0 + 64u;
            const uint32_t o0 = (int)k0 < kend ? k0 : kOob, o1 = (int)k1 < kend ? k1 : kOob;
            w[u] = join8(buf_load16(wr, woff + o0, 0), buf_load16(wr, woff + o1, 0));
#pragma unroll
            for (int t = 0; t < TF; ++t) {
                a[u][t] = join8(buf_load16(ar, aoff[t] + o0, 0), buf_load16(ar, aoff[t] + o1, 0));
                s[u][t] = buf_load_f32(sr, kb < KB ? soff[t] + (uint32_t)kb * 4u : kOob, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // past the last block both scales are zero (an infinite one times zero is none)
            const int kb = kbase + u * kstep;
            const float ws = kb < KB ? sw[min(kb, KB - 1)] : 0.0f;
#pragma unroll
            for (int t = 0; t < TF; ++t) {
                const f32x4_t d = mfma_fp8<kExact>(w[u], a[u][t]);
                const float c = s[u][t] * ws;
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[t][j] = fmaf(c, d[j], acc[t][j]);
            }
        }
    }
}

constexpr int kSkThreads = 512, kSkWaves = kSkThreads / kWave;

// Dense product: a workgroup computes 16 outputs of 16 TF rows; wave v takes the blocks v, v + 8, ... of the inputs.
template <int TF, bool kExact>
__global__ __launch_bounds__(kSkThreads) void fp8_skinny_kernel(const Fp8Dense p) {
    __shared__ f32x4_t part[kSkWaves][TF][kWave];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const int nt = (p.N + 15) / 16, n0 = blockIdx.x % nt * 16, m0 = blockIdx.x / nt * 16 * TF;
    const int KB = fp8_blocks(p.K);
    const __amdgpu_buffer_rsrc_t wr =
        fp8_rsrc(p.w + (size_t)n0 * p.ldw, (uint32_t)((min(p.N - n0, 16) - 1) * p.ldw + p.K));
    const int mr = min(p.M - m0, 16 * TF);
    const __amdgpu_buffer_rsrc_t ar = fp8_rsrc(p.a + (size_t)m0 * p.lda, (uint32_t)((mr - 1) * p.lda + p.K));
    const __amdgpu_buffer_rsrc_t sr = fp8_rsrc(p.sa + (size_t)m0 * KB, (uint32_t)mr * (uint32_t)KB * 4u);
    const float* sw = p.sw + (size_t)(n0 / 128) * KB;
    uint32_t aoff[TF], soff[TF];
#pragma unroll
    for (int t = 0; t < TF; ++t) {
        aoff[t] = (uint32_t)(16 * t + l16) * (uint32_t)p.lda;
        soff[t] = (uint32_t)(16 * t + l16) * (uint32_t)KB * 4u;
        if (16 * t + l16 >= mr) soff[t] = kOob;
    }
    f32x4_t acc[TF];
#pragma unroll
    for (int t = 0; t < TF; ++t) acc[t] = f32x4_t{};
    fp8_wave_product<TF, kExact>(acc, wr, (uint32_t)l16 * (uint32_t)p.ldw, ar, aoff, sr, soff, sw, wv, kSkWaves, KB, p.K, g);
#pragma unroll
    for (int t = 0; t < TF; ++t) part[wv][t][lane] = acc[t];
    __syncthreads();
    // joined in the order of the waves
    for (int t = wv; t < TF; t += kSkWaves) {
        f32x4_t v = part[0][t][lane];
#pragma unroll
        for (int i = 1; i < kSkWaves; ++i) v += part[i][t][lane];
        const int m = 16 * t + l16, n = n0 + 4 * g;
        if (m < mr && n < p.N) {
            char* row = static_cast<char*>(p.y) + (m0 + m) * p.ldy * (p.out_f32 ? 4 : 2);
            fp8_store4(row, p.out_f32, n, p.N, p.vec && n + 3 < p.N, v);
        }
    }
}

long fp8_skinny_workgroups(int M, int N) { return ((long)N + 15) / 16 * (M <= 16 ? 1 : ((long)M + 31) / 32); }

hipError_t launch_fp8_skinny(const Fp8Dense& p, hipStream_t s) {
    const dim3 grid((unsigned)fp8_skinny_workgroups(p.M, p.N)), block(kSkThreads);
    if (p.M <= 16) {
        if (p.out_f32) hipLaunchKernelGGL((fp8_skinny_kernel<1, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((fp8_skinny_kernel<1, false>), grid, block, 0, s, p);
    } else {
        if (p.out_f32) hipLaunchKernelGGL((fp8_skinny_kernel<2, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((fp8_skinny_kernel<2, false>), grid, block, 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace moe
