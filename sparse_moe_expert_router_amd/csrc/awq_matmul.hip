// Product of few bf16 rows with one AWQ matrix (4-bit codes, zeros and fp16
// scales per group of 32, 64 or 128 inputs, in GEMM packing):
//   y[m][n] = sum_g s[g][n] * sum_{i in g} x[m][i] (q[i][n] - z[g][n])
//
// Bound by the codes' bytes.  A word holds one input of 8 columns, so a lane
// that reads the words of 8 consecutive inputs holds, for each of the word's 8
// columns, 8 inputs: the operand of the 16 x 16 x 32 bf16 MFMA for that
// column, with the four 16-lane groups of a wave covering the 32 inputs of a
// step and the 16 lanes of a group 16 words, that is 128 columns.  Two v_perm
// bring the halves of two inputs' words together, then a shift and a v_and_or
// make the exact bf16 pair 16 + q of one column.  The product with 16 + q is
// exact up to fp32 sums, and
//   sum x (q - z) = sum x (16 + q) - (16 + z) sum x
// with sum x from one more MFMA whose second operand is ones, so it lies in
// the lanes as the products do.  (128 + q would save a shift, at eight times
// the cancellation.)  The scale is applied in fp32.
//
// The 8 waves of a workgroup take consecutive runs of inputs of the same columns
// and add their sums through LDS in a fixed order; where the columns alone do
// not fill the card the inputs are split over workgroups too, whose fp32 sums
// a second kernel adds.
#include "kernels.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kWaves = 8;
constexpr int kAhead = 4;   // steps of 32 inputs whose loads are in flight
constexpr int kTile = 128;  // columns of 16 words

struct Awq {
    const uint16_t* x;
    int64_t ldx;
    const uint32_t* qw;
    const uint32_t* qz;
    const uint16_t* sc;
    int M, N, K, gshift;  // group = 32 << gshift
    int f32;
    void* y;
    int64_t ldy;
    float* part;  // nullptr: y itself
};

__device__ __forceinline__ int nibble_column(int j) { return (j & 3) * 2 + (j >> 2); }  // 0,2,4,6,1,3,5,7

__device__ __forceinline__ void put(const Awq& a, int64_t m, int n, float v) {
    if (a.f32) static_cast<float*>(a.y)[m * a.ldy + n] = v;
    else static_cast<uint16_t*>(a.y)[m * a.ldy + n] = (uint16_t)f32_to_bf16_bits(v);
}

// The loads of one step.
template <int MT>
struct Step {
    uint32_t w[8];
    uint32_t z;
    uint4 s;
    uint4 x[MT];
};

template <int MT>
__global__ __launch_bounds__(64 * kWaves) void awq_matmul_kernel(Awq a) {
    __shared__ __align__(16) f32x4_t red[kWaves][8][64];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int kq = lane / 16, n16 = lane % 16;
    const int n8 = a.N / 8;
    const int m0 = blockIdx.z * 16 * MT;
    const int word = blockIdx.x * 16 + n16;
    const int wl = word < n8 ? word : n8 - 1;  // lanes past the last word read it again and store nothing

    // this wave's groups
    const int64_t groups = a.K >> (5 + a.gshift);
    const int slices = gridDim.y * kWaves, slice = blockIdx.y * kWaves + wave;
    const int first = (int)(groups * slice / slices) << a.gshift;
    const int end = (int)(groups * (slice + 1) / slices) << a.gshift;  // steps [first, end)

    const uint16_t* xr[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = m0 + 16 * t + n16;
        xr[t] = a.x + (int64_t)(m < a.M ? m : a.M - 1) * a.ldx + 8 * kq;
    }
    const uint32_t row0 = (uint32_t)(8 * kq) * n8 + wl;

    auto fetch = [&](int step, Step<MT>& st) {
        const uint32_t* q = a.qw + (int64_t)step * 32 * n8;
#pragma unroll
        for (int i = 0; i < 8; ++i) st.w[i] = __builtin_nontemporal_load(q + row0 + (uint32_t)i * n8);
        const int64_t g = step >> a.gshift;
        st.z = a.qz[g * n8 + wl];
        st.s = *reinterpret_cast<const uint4*>(a.sc + (g * n8 + wl) * 8);
#pragma unroll
        for (int t = 0; t < MT; ++t) st.x[t] = *reinterpret_cast<const uint4*>(xr[t] + (int64_t)step * 32);
    };

    f32x4_t acc[MT][8];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t][j] = f32x4_t(0.0f);
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u));
    const f32x4_t zero = f32x4_t(0.0f);

    if (first < end) {
        Step<MT> ring[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) fetch(first + u < end ? first + u : end - 1, ring[u]);
        for (int s0 = first; s0 < end; s0 += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (s0 + u < end) {
                    const Step<MT>& st = ring[u];
                    f32x4_t sx[MT];
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        sx[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, st.x[t]), ones, zero, 0, 0, 0);
                    uint32_t lo[4], hi[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        lo[p] = __builtin_amdgcn_perm(st.w[2 * p + 1], st.w[2 * p], 0x05040100u);
                        hi[p] = __builtin_amdgcn_perm(st.w[2 * p + 1], st.w[2 * p], 0x07060302u);
                    }
                    const uint32_t sw[4] = {st.s.x, st.s.y, st.s.z, st.s.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t b[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const uint32_t v = j < 4 ? lo[p] : hi[p];
                            b[p] = and_or(j % 4 == 0 ? v << 3 : v >> (4 * (j % 4) - 3), 0x00780078u, 0x41804180u);
                        }
                        const bf16x8_t bj = __builtin_bit_cast(bf16x8_t, make_uint4(b[0], b[1], b[2], b[3]));
                        // 16 + z as fp32
                        const float z = __uint_as_float(and_or(j < 5 ? st.z << (19 - 4 * j) : st.z >> (4 * j - 19), 0x00780000u, 0x41800000u));
                        const int c = nibble_column(j);
                        const float sc = f16_to_f32((sw[c / 2] >> (16 * (c % 2))) & 0xFFFFu);
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const f32x4_t d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, st.x[t]), bj, zero, 0, 0, 0);
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(sc, fmaf(-z, sx[t][i], d[i]), acc[t][j][i]);
                        }
                    }
                }
                fetch(s0 + u + kAhead < end ? s0 + u + kAhead : end - 1, ring[u]);
            }
        }
    }

    // the waves' sums: thread (j, lane) adds column nibble j of the lane's word, four rows
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t) __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) red[wave][j][lane] = acc[t][j];
        __syncthreads();
        f32x4_t v = red[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][wave][lane];
        const int n = 8 * word + nibble_column(wave);
        if (word < n8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + 16 * t + 4 * kq + i;
                if (m < a.M) {
                    if (a.part) a.part[((int64_t)blockIdx.y * a.M + m) * a.N + n] = v[i];
                    else put(a, m, n, v[i]);
                }
            }
        }
    }
}

// y = the `splits` partial sums, in order.
__global__ __launch_bounds__(256) void awq_sum_kernel(Awq a, int splits) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)a.M * a.N;
    if (i >= n) return;
    float v = 0.0f;
    for (int s = 0; s < splits; ++s) v += a.part[s * n + i];
    put(a, i / a.N, (int)(i % a.N), v);
}

int row_tiles(int M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }  // 16-row tiles of a workgroup

int awq_splits(int M, int N, int K, int group) {
    const int mt = row_tiles(M);
    const int64_t tiles = (int64_t)((N + kTile - 1) / kTile) * ((M + 16 * mt - 1) / (16 * mt));
    const int64_t fill = 512 / tiles;                    // workgroups that fill the card twice
    const int64_t deep = K / group / kWaves / (256 / group);  // at least 256 inputs a wave
    int64_t s = fill < deep ? fill : deep;
    return s < 2 ? 1 : (int)s;
}

}  // namespace

size_t awq_matmul_ws_bytes(int M, int N, int K, int group) {
    const int s = awq_splits(M, N, K, group);
    return s > 1 ? (size_t)s * M * N * sizeof(float) : 0;
}

hipError_t launch_awq_matmul(const uint16_t* x, int64_t ldx, const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                             int M, int N, int K, int group, int out_f32, void* y, int64_t ldy, void* ws, hipStream_t s) {
    Awq a{};
    a.x = x; a.ldx = ldx;
    a.qw = reinterpret_cast<const uint32_t*>(qweight);
    a.qz = reinterpret_cast<const uint32_t*>(qzeros);
    a.sc = scales;
    a.M = M; a.N = N; a.K = K; a.gshift = group == 32 ? 0 : group == 64 ? 1 : 2;
    a.f32 = out_f32; a.y = y; a.ldy = ldy;
    const int splits = awq_splits(M, N, K, group);
    a.part = splits > 1 ? static_cast<float*>(ws) : nullptr;
    const int mt = row_tiles(M);
    const dim3 grid((N + kTile - 1) / kTile, splits, (M + 16 * mt - 1) / (16 * mt)), block(64 * kWaves);
    if (mt == 1) hipLaunchKernelGGL((awq_matmul_kernel<1>), grid, block, 0, s, a);
    else if (mt == 2) hipLaunchKernelGGL((awq_matmul_kernel<2>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((awq_matmul_kernel<4>), grid, block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || splits == 1) return e;
    const int64_t n = (int64_t)M * N;
    hipLaunchKernelGGL(awq_sum_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a, splits);
    return hipGetLastError();
}

}  // namespace moe
