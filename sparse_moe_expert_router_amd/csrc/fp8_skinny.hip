// W8A8 products for few rows: E4M3 codes on both sides, fp32 scales per 128
// inputs (rows) and per 128 x 128 block (weights), gfx950's 16 x 16 x 128 FP8
// MFMA (fp32 outputs: the bf16 MFMA on widened codes, see mfma_fp8).  One
// call of it covers one block of 128 inputs of 16 outputs x 16 rows; its
// result is multiplied by the two scales and
// added to an fp32 accumulator:
//   y[m][n] += (sa[m][kb] * sw[n / 128][kb]) * sum_i a[m][i] w[n][i].
// The weights are the MFMA's row operand, so a lane ends up with four
// neighbouring outputs of one row.
//
// With few rows the weights' bytes bound the call.  They go from memory
// straight into registers, each byte once per row tile; rows are read from
// the caches.  The work is cut into 16 outputs a wave; a dense product with
// its few outputs also splits the inputs over the 8 waves of a workgroup and
// joins them through LDS in a fixed order.
#include "fp8.h"
#include "ffn_internal.h"
#include "fp8_internal.h"

namespace moe {

// One wave's product of NW blocks of 16 weight rows with TF groups of 16
// activation rows over blocks kb0, kb0 + kstep, ... < KB of 128 inputs.
// wr / ar: buffers whose rows past the end read as zero; woff / aoff: the
// lane's byte offset of its row; kend: bytes of a row (a multiple of 16).
template <int NW, int TF, bool kExact>
__device__ __forceinline__ void fp8_wave_product(f32x4_t (&acc)[NW][TF], const __amdgpu_buffer_rsrc_t (&wr)[NW],
                                                 uint32_t woff, __amdgpu_buffer_rsrc_t ar, const uint32_t (&aoff)[TF],
                                                 __amdgpu_buffer_rsrc_t sr, const uint32_t (&soff)[TF],
                                                 const float* const (&sw)[NW], int kb0, int kstep, int KB, int kend,
                                                 int g) {
    constexpr int U = NW + TF <= 2 ? 5 : 4;  // blocks loaded before the first is used
    for (int kbase = kb0; kbase < KB; kbase += U * kstep) {
        i32x8_t w[U][NW], a[U][TF];
        float s[U][TF];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // a lane group's 32 inputs: pieces g and g + 4 of the block's
            // eight.  Past the row's end both sides and the scales read zero.
            const int kb = kbase + u * kstep;
            const uint32_t k0 = (uint32_t)kb * 128u + 16u * (uint32_t)g, k1 = k0 + 64u;
            const uint32_t o0 = (int)k0 < kend ? k0 : kOob, o1 = (int)k1 < kend ? k1 : kOob;
#pragma unroll
            for (int i = 0; i < NW; ++i)
                w[u][i] = join8(buf_load16(wr[i], woff + o0, 0), buf_load16(wr[i], woff + o1, 0));
#pragma unroll
            for (int t = 0; t < TF; ++t) {
                a[u][t] = join8(buf_load16(ar, aoff[t] + o0, 0), buf_load16(ar, aoff[t] + o1, 0));
                s[u][t] = buf_load_f32(sr, kb < KB ? soff[t] + (uint32_t)kb * 4u : kOob, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = min(kbase + u * kstep, KB - 1);
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int t = 0; t < TF; ++t) {
                    const f32x4_t d = mfma_fp8<kExact>(w[u][i], a[u][t]);
                    const float c = s[u][t] * sw[i][kb];
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][t][j] = fmaf(c, d[j], acc[i][t][j]);
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
    const __amdgpu_buffer_rsrc_t wr[1] = {
        fp8_rsrc(p.w + (size_t)n0 * p.ldw, (uint32_t)((min(p.N - n0, 16) - 1) * p.ldw + p.K))};
    const int mr = min(p.M - m0, 16 * TF);
    const __amdgpu_buffer_rsrc_t ar = fp8_rsrc(p.a + (size_t)m0 * p.lda, (uint32_t)((mr - 1) * p.lda + p.K));
    const __amdgpu_buffer_rsrc_t sr = fp8_rsrc(p.sa + (size_t)m0 * KB, (uint32_t)mr * (uint32_t)KB * 4u);
    const float* const sw[1] = {p.sw + (size_t)(n0 / 128) * KB};
    uint32_t aoff[TF], soff[TF];
#pragma unroll
    for (int t = 0; t < TF; ++t) {
        aoff[t] = (uint32_t)(16 * t + l16) * (uint32_t)p.lda;
        soff[t] = (uint32_t)(16 * t + l16) * (uint32_t)KB * 4u;
        if (16 * t + l16 >= mr) soff[t] = kOob;
    }
    f32x4_t acc[1][TF];
#pragma unroll
    for (int t = 0; t < TF; ++t) acc[0][t] = f32x4_t{};
    fp8_wave_product<1, TF, kExact>(acc, wr, (uint32_t)l16 * (uint32_t)p.ldw, ar, aoff, sr, soff, sw, wv, kSkWaves, KB, p.K, g);
#pragma unroll
    for (int t = 0; t < TF; ++t) part[wv][t][lane] = acc[0][t];
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

// Rows of tile `i` of the table: expert, first row, end row (at most 16 rows).
__device__ __forceinline__ bool a8_tile(const Fp8Ffn& p, int i, int* e, int* r0, int* r1) {
    if (i >= p.tiles[0]) return false;
    *e = p.tiles[1 + 3 * i];
    *r0 = p.tiles[2 + 3 * i];
    *r1 = min(p.tiles[3 + 3 * i], p.P);
    return *r0 >= 0 && *r0 < *r1;
}

// Gate and up of 128 inner columns for one tile of at most 16 rows, SwiGLU,
// and the quantisation of its product for the down pass: wave v holds columns
// 16 v .. +15 of the group, so the group's largest magnitude is a maximum
// over the lanes of a row and over the waves.
__global__ __launch_bounds__(kSkThreads) void fp8_skinny_gateup_kernel(const Fp8Ffn p) {
    __shared__ uint32_t amax[kSkWaves][16];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    int e, r0, r1;
    const int nf = p.F / 128, fg = blockIdx.x % nf;
    if (!a8_tile(p, blockIdx.x / nf, &e, &r0, &r1)) return;
    const int f0 = fg * 128 + wv * 16, KB = p.H / 128;
    const size_t wbase = ((size_t)e * p.F + f0) * p.H;
    const __amdgpu_buffer_rsrc_t wr[2] = {fp8_rsrc(p.gate + wbase, 16u * (uint32_t)p.H),
                                          fp8_rsrc(p.up + wbase, 16u * (uint32_t)p.H)};
    const size_t sbase = ((size_t)e * (p.F / 128) + fg) * KB;
    const float* const sw[2] = {p.sgate + sbase, p.sup + sbase};
    const int row = min(r0 + l16, r1 - 1);
    const int tok = p.sorted_pair ? min(max(p.sorted_pair[row] / p.k, 0), p.T - 1) : row;
    const __amdgpu_buffer_rsrc_t ar = fp8_rsrc(p.xq, (uint32_t)p.T * (uint32_t)p.H);
    const __amdgpu_buffer_rsrc_t sr = fp8_rsrc(p.xs, (uint32_t)p.T * (uint32_t)KB * 4u);
    const uint32_t aoff[1] = {(uint32_t)tok * (uint32_t)p.H}, soff[1] = {(uint32_t)tok * (uint32_t)KB * 4u};
    f32x4_t acc[2][1] = {{f32x4_t{}}, {f32x4_t{}}};
    fp8_wave_product<2, 1, false>(acc, wr, (uint32_t)l16 * (uint32_t)p.H, ar, aoff, sr, soff, sw, 0, 1, KB, p.H, g);
    float h[4];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = silu(acc[0][0][j]) * acc[1][0][j];
        m = max(m, abs_bits(h[j]));
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
    if (g == 0) amax[wv][l16] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSkWaves; ++i) m = max(m, amax[i][l16]);
    const float s = fp8_scale(m);
    if (r0 + l16 < r1) {
        *reinterpret_cast<uint32_t*>(p.hq + (size_t)row * p.F + f0 + 4 * g) = fp8_pack4(h[0], h[1], h[2], h[3], s);
        if (wv == 0 && g == 0) p.hs[(size_t)row * (p.F / 128) + fg] = s;
    }
}

// Down projection of one tile of at most 16 rows: a workgroup computes 128
// outputs, wave v 16 of them.
__global__ __launch_bounds__(kSkThreads) void fp8_skinny_down_kernel(const Fp8Ffn p) {
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    int e, r0, r1;
    const int nh = p.H / 128, nb = blockIdx.x % nh;
    if (!a8_tile(p, blockIdx.x / nh, &e, &r0, &r1)) return;
    const int n0 = nb * 128 + wv * 16, KB = p.F / 128;
    const __amdgpu_buffer_rsrc_t wr[1] = {fp8_rsrc(p.down + ((size_t)e * p.H + n0) * p.F, 16u * (uint32_t)p.F)};
    const float* const sw[1] = {p.sdown + ((size_t)e * (p.H / 128) + nb) * KB};
    const __amdgpu_buffer_rsrc_t ar = fp8_rsrc(p.hq + (size_t)r0 * p.F, (uint32_t)(r1 - r0) * (uint32_t)p.F);
    const __amdgpu_buffer_rsrc_t sr = fp8_rsrc(p.hs + (size_t)r0 * KB, (uint32_t)(r1 - r0) * (uint32_t)KB * 4u);
    const int row = min(l16, r1 - r0 - 1);
    const uint32_t aoff[1] = {(uint32_t)row * (uint32_t)p.F}, soff[1] = {(uint32_t)row * (uint32_t)KB * 4u};
    f32x4_t acc[1][1] = {{f32x4_t{}}};
    fp8_wave_product<1, 1, false>(acc, wr, (uint32_t)l16 * (uint32_t)p.F, ar, aoff, sr, soff, sw, 0, 1, KB, p.F, g);
    if (r0 + l16 < r1)
        fp8_store4(static_cast<char*>(p.rows) + (size_t)(r0 + l16) * p.H * (p.out_f32 ? 4 : 2), p.out_f32, n0 + 4 * g,
               p.H, true, acc[0][0]);
}

hipError_t launch_fp8_skinny(const Fp8Dense& p, hipStream_t s) {
    const int nt = (p.N + 15) / 16;
    const int mt = p.M <= 16 ? 1 : (p.M + 31) / 32;
    const dim3 grid(nt * mt), block(kSkThreads);
    if (p.M <= 16) {
        if (p.out_f32) hipLaunchKernelGGL((fp8_skinny_kernel<1, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((fp8_skinny_kernel<1, false>), grid, block, 0, s, p);
    } else {
        if (p.out_f32) hipLaunchKernelGGL((fp8_skinny_kernel<2, true>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((fp8_skinny_kernel<2, false>), grid, block, 0, s, p);
    }
    return hipGetLastError();
}

hipError_t launch_fp8_skinny_ffn(const Fp8Ffn& p, int max_tiles, hipStream_t s) {
    hipLaunchKernelGGL(fp8_skinny_gateup_kernel, dim3(p.F / 128 * max_tiles), dim3(kSkThreads), 0, s, p);
    hipLaunchKernelGGL(fp8_skinny_down_kernel, dim3(p.H / 128 * max_tiles), dim3(kSkThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace moe
