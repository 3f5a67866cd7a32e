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
// one row after another; short rows take 16 lanes.  (32768 x 2560, residual and
// codes: 107 us, 5.5 TB/s; the gradients 125 us, 5.4 TB/s; a large copy runs
// at 5.2.)
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

// A row's threads: the workgroup (kL = 64), or 16 lanes (kL = 16, for rows of up
// to 256 values) with 16 rows to a workgroup.
constexpr int kRowsOf16 = 16;  // rows of a workgroup with kL = 16
template <int kL>
struct Team {
    int n, t, team, teams;  // threads of a row, this one among them; rows in work, this one among them
    __device__ __forceinline__ Team() {
        n = kL == 16 ? 16 : blockDim.x;
        t = kL == 16 ? threadIdx.x % 16 : threadIdx.x;
        team = kL == 16 ? threadIdx.x / 16 : 0;
        teams = kL == 16 ? kRowsOf16 : 1;
    }
    __device__ __forceinline__ float sum(float v, float* red) const {
        return kL == 16 ? sum16_f32(v) : row_sum(v, red, n / kWave);
    }
};

// Eight values as they lie in memory: a row's loads are all issued before the
// first is converted (with the types known at run time only they are not: 32768 x
// 2560 to codes 107 -> 126 us).
template <bool kF32>
struct Raw8 {
    uint4 v[kF32 ? 2 : 1];
};
template <bool kF32>
__device__ __forceinline__ Raw8<kF32> raw8(const void* p, int64_t i) {
    Raw8<kF32> r;
    if constexpr (kF32) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        r.v[0] = s[0];
        r.v[1] = s[1];
    } else {
        r.v[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    }
    return r;
}
template <bool kF32>
__device__ __forceinline__ f32x8_t values(const Raw8<kF32>& r) {
    return load8(r.v, 0, kF32);
}

// kX: x is fp32; kR: 0 no residual, 1 bf16, 2 fp32.  The next row's loads are on
// their way while a row is summed and written.
template <int kL, int C, bool kX, int kR>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
    __shared__ float red[2][kMaxWaves];
    const Team<kL> m;
    const int n = m.n, t = m.t, nb = fp8_blocks(a.H);
    const int64_t step = (int64_t)gridDim.x * m.teams;
    struct Row {
        Raw8<kX> x[C];
        Raw8<kR == 2> r[C];
    } cur, next;
    auto fetch = [&](int64_t row, Row& f) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (c * n + t);
            if (i >= a.H || row >= a.T) continue;
            f.x[c] = raw8<kX>(a.x, row * a.ldx + i);
            if constexpr (kR != 0) f.r[c] = raw8<kR == 2>(a.res, row * a.ldr + i);
        }
    };
    int64_t first = (int64_t)blockIdx.x * m.teams;
    fetch(first + m.team, cur);
    // with the offset 1 the gain's sum is part of a multiply-add, and costs no rounding
    const bool one = a.offset == 1.0f;
    f32x8_t gain[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        gain[c] = 8 * (c * n + t) < a.H ? load8(a.w, 8 * (c * n + t), a.w_f32) : f32x8_t(0.0f);
        if (!one) gain[c] += a.offset;
    }
    int flip = 0;
    // (the lanes of a wave stay together: rows past the last one are empty)
    for (; first < a.T; first += step, flip ^= 1) {
        const int64_t row = first + m.team;
        if (first + step < a.T) fetch(row + step, next);
        bool in[C];
        f32x8_t s[C];
        float sq = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (c * n + t);
            in[c] = i < a.H && row < a.T;
            s[c] = f32x8_t(0.0f);
            if (in[c]) {
                s[c] = values(cur.x[c]);
                if constexpr (kR != 0) {
                    s[c] += values(cur.r[c]);
                    if constexpr (kR == 1) {
                        const uint4 q = pack8(s[c]);
                        s[c] = load8(&q, 0, 0);
                    }
                    store8(a.res_out, row * a.ldro + i, kR == 2, s[c]);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fmaf(s[c][j], s[c][j], sq);
        }
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(m.sum(sq, red[flip]), (float)a.H) + a.eps));
        if (a.rstd && t == 0 && row < a.T) a.rstd[row] = r;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (c * n + t);
            f32x8_t v = s[c] * r;
            if (one) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], gain[c][j], v[j]);
            } else {
                v *= gain[c];
            }
            if (a.y && in[c]) store8(a.y, row * a.ldy + i, 0, v);
            if (a.codes) {
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, in[c] ? abs_bits(v[j]) : 0u);
                const float sc = fp8_scale(max16_u32(top));
                const Fp8Div d = fp8_div(in[c] ? sc : 1.0f);
                if (in[c]) {
                    const uint2 q = make_uint2(fp8_pack4(v[0], v[1], v[2], v[3], d), fp8_pack4(v[4], v[5], v[6], v[7], d));
                    *reinterpret_cast<uint2*>(a.codes + row * a.H + i) = q;
                    if (t % 16 == 0) a.scales[row * nb + i / kFp8Block] = sc;
                }
            }
        }
        cur = next;
    }
}

// Four values as they lie in memory, and as they are.
template <bool kF32>
struct Raw4 {
    uint32_t v[kF32 ? 4 : 2];
};
template <bool kF32>
__device__ __forceinline__ Raw4<kF32> raw4(const void* p, int64_t i) {
    if constexpr (kF32) {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        return {{q.x, q.y, q.z, q.w}};
    } else {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
        return {{q.x, q.y}};
    }
}
template <bool kF32>
__device__ __forceinline__ f32x4_t values4(const Raw4<kF32>& r) {
    f32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (kF32) v[j] = __uint_as_float(r.v[j]);
        else v[j] = __uint_as_float(j % 2 ? r.v[j / 2] & 0xFFFF0000u : r.v[j / 2] << 16);
    }
    return v;
}

// dw of the 32 columns at `first`, from all rows: thread (p0, q) takes rows p0,
// p0 + n, .. of columns 4q..4q+3, eight rows' loads on their way at a time.  The
// workgroup has 16 waves at most, an even number of them.
template <bool kY, bool kS>
__device__ __forceinline__ void norm_dw_columns(const NormBwdArgs& a, int first) {
    __shared__ __align__(16) f32x4_t red[128][8];
    const int q = threadIdx.x % 8, p0 = threadIdx.x / 8, n = blockDim.x / 8, col = first + 4 * q;
    f32x4_t v = f32x4_t(0.0f);
    if (col < a.H) {
        for (int64_t p = p0; p < a.T; p += 8 * n) {
            Raw4<kY> dy[8];
            Raw4<kS> s[8];
            float r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t row = p + i * n < a.T ? p + i * n : p;
                dy[i] = raw4<kY>(a.dy, row * a.ldy + col);
                s[i] = raw4<kS>(a.s, row * a.lds + col);
                r[i] = a.rstd[row];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (p + i * n < a.T) v += values4(dy[i]) * (values4(s[i]) * r[i]);
        }
    }
    red[p0][q] = v;
    __syncthreads();
    if (p0 < 16) {
        for (int i = p0 + 16; i < n; i += 16) v += red[i][q];
        red[p0][q] = v;
    }
    __syncthreads();
    if (p0 == 0 && col < a.H) {
#pragma unroll
        for (int i = 1; i < 16; ++i) v += red[i][q];
#pragma unroll
        for (int j = 0; j < 4; ++j) a.dw[col + j] = v[j];
    }
}

// kY: dy is fp32; kS: s, dres and dx are.  `part` gets one row of sums of dy h
// from each workgroup; with kOne the first `columns` workgroups make dw instead.
template <int kL, int C, bool kY, bool kS, bool kOne>
__global__ __launch_bounds__(kL == 16 ? 16 * kRowsOf16 : 1024) void norm_bwd_kernel(NormBwdArgs a, float* __restrict__ part, int columns) {
    if constexpr (kOne) {
        if ((int)blockIdx.x < columns) {
            norm_dw_columns<kY, kS>(a, blockIdx.x * 32);
            return;
        }
    }
    __shared__ float red[2][kMaxWaves];
    constexpr bool kEarly = C == 1 || !kS;  // dres is loaded with the rest (two fp32 pieces would not fit the registers)
    const Team<kL> m;
    const int group = kOne ? blockIdx.x - columns : blockIdx.x, groups = kOne ? gridDim.x - columns : gridDim.x;
    const int n = m.n, t = m.t;
    f32x8_t gain[C], dw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = 8 * (c * n + t);
        gain[c] = i < a.H ? load8(a.w, i, a.w_f32) + a.offset : f32x8_t(0.0f);
        dw[c] = f32x8_t(0.0f);
    }
    int flip = 0;
    for (int64_t first = (int64_t)group * m.teams; first < a.T; first += (int64_t)groups * m.teams, flip ^= 1) {
        const int64_t row = first + m.team;
        const float r = row < a.T ? a.rstd[row] : 0.0f;
        bool in[C];
        Raw8<kS> rs[C], rd[C];
        Raw8<kY> ry[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (c * n + t);
            in[c] = i < a.H && row < a.T;
            if (!in[c]) continue;
            rs[c] = raw8<kS>(a.s, row * a.lds + i);
            ry[c] = raw8<kY>(a.dy, row * a.ldy + i);
            if (kEarly && a.dres) rd[c] = raw8<kS>(a.dres, row * a.lddr + i);
        }
        f32x8_t h[C], u[C];
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            h[c] = u[c] = f32x8_t(0.0f);
            if (in[c]) {
                h[c] = values(rs[c]) * r;
                const f32x8_t dy = values(ry[c]);
                if constexpr (!kOne) dw[c] += dy * h[c];
                u[c] = dy * gain[c];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) dot = fmaf(u[c][j], h[c][j], dot);
        }
        const float mean = __fdiv_rn(m.sum(dot, red[flip]), (float)a.H);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = 8 * (c * n + t);
            if (!in[c]) continue;
            f32x8_t d = (u[c] - h[c] * mean) * r;
            if (a.dres) d += values(kEarly ? rd[c] : raw8<kS>(a.dres, row * a.lddr + i));
            store8(a.dx, row * a.lddx + i, kS, d);
        }
    }
    if constexpr (kOne) return;
    if constexpr (kL == 16) {
        // the workgroup's 16 rows of sums, in order
        __shared__ __align__(16) f32x8_t sums[C][kRowsOf16][16];
#pragma unroll
        for (int c = 0; c < C; ++c) sums[c][m.team][t] = dw[c];
        __syncthreads();
        if (m.team != 0) return;
#pragma unroll
        for (int c = 0; c < C; ++c)
            for (int i = 1; i < kRowsOf16; ++i) dw[c] += sums[c][i][t];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = 8 * (c * n + t);
        if (i < a.H) store8(part, (int64_t)blockIdx.x * a.H + i, 1, dw[c]);
    }
}

// dw [H] = sum of the `parts` partial rows: 32 columns (whole lines) a workgroup.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ part, int parts, int H, float* __restrict__ dw) {
    __shared__ __align__(16) f32x4_t red[128][8];
    const int q = threadIdx.x % 8, p0 = threadIdx.x / 8;
    const int col = blockIdx.x * 32 + 4 * q;
    f32x4_t v = col < H ? sum_rows(part + col, parts, H, p0) : f32x4_t(0.0f);
    red[p0][q] = v;
    __syncthreads();
    v = sum_128(v, red, p0, q);
    if (p0 == 0 && col < H) {
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[col + j] = v[j];  // (dw has no more than its element's alignment)
    }
}

namespace {

struct Plan {
    int lanes, c, block, grid;
};

// Rows of up to 256 values take 16 lanes (32768 x 64: 8.6 -> 4.6 us).  Longer ones take whole waves, with c pieces a
// thread: two where 16 waves of one would not do, or as asked.
Plan shape(int H, bool two) {
    Plan p;
    p.lanes = H <= 256 ? 16 : 64;
    p.c = p.lanes == 16 ? (H <= 128 ? 1 : 2) : two || H > 8 * 64 * kMaxWaves ? 2 : 1;
    p.block = p.lanes == 16 ? 16 * kRowsOf16 : (H + 512 * p.c - 1) / (512 * p.c) * 64;
    p.grid = 0;
    return p;
}
int workgroups(const Plan& p, int T, int most) {
    const int rows = p.lanes == 16 ? kRowsOf16 : 1, need = (int)(((int64_t)T + rows - 1) / rows);
    return need < most ? need : most;
}

// Many rows take two pieces a thread (32768 x 2560 to codes: 110 -> 107 us; one row 2.7 against 2.9), and up to eight
// rounds of the workgroups that the card holds (two rounds 116).
Plan norm_plan(int T, int H) {
    Plan p = shape(H, T >= 8192);
    p.grid = workgroups(p, T, 256 * (2048 / p.block) * 8);
    return p;
}

// Each workgroup writes one partial row of dw, so there are no more than keep the memory busy, about ten waves a
// compute unit (32768 x 2560: 512 workgroups 125 us, 1024 154; 32768 x 640: 512 85, 1280 53, 1536 53).
Plan bwd_plan(int T, int H) {
    Plan p = shape(H, false);
    if (p.lanes == 64 && p.c == 2) p.block = (p.block + 127) / 128 * 128;  // (as with one launch, for the same bits of dx)
    const int waves = p.block / 64;
    p.grid = workgroups(p, T, 256 * ((10 + waves - 1) / waves));
    return p;
}

template <int kL, int C>
void run_norm(const NormArgs& a, const Plan& p, hipStream_t s) {
    const dim3 grid(p.grid), block(p.block);
#define MOE_NORM(kX, kR) hipLaunchKernelGGL((norm_kernel<kL, C, kX, kR>), grid, block, 0, s, a)
    if (a.x_f32) {
        if (!a.res) MOE_NORM(true, 0);
        else if (a.r_f32) MOE_NORM(true, 2);
        else MOE_NORM(true, 1);
    } else {
        if (!a.res) MOE_NORM(false, 0);
        else if (a.r_f32) MOE_NORM(false, 2);
        else MOE_NORM(false, 1);
    }
#undef MOE_NORM
}

template <int kL, int C, bool kOne>
void run_norm_bwd(const NormBwdArgs& a, const Plan& p, float* part, hipStream_t s) {
    const int columns = kOne ? (a.H + 31) / 32 : 0;
    const dim3 grid(p.grid + columns), block(p.block);
#define MOE_NORM_BWD(kY, kS) hipLaunchKernelGGL((norm_bwd_kernel<kL, C, kY, kS, kOne>), grid, block, 0, s, a, part, columns)
    if (a.y_f32) {
        if (a.s_f32) MOE_NORM_BWD(true, true);
        else MOE_NORM_BWD(true, false);
    } else {
        if (a.s_f32) MOE_NORM_BWD(false, true);
        else MOE_NORM_BWD(false, false);
    }
#undef MOE_NORM_BWD
}

// Few rows: dw is made by workgroups of its own, which read s and dy once more, beside those that make dx, in one launch
// (515 x 688 fp32: 7.8 -> 5.3 us, 515 x 8192 17.8 -> 15.5, 1024 x 8192 22.6 -> 25.6).  dx may then lie on neither s nor dy.
bool one_launch(const NormBwdArgs& a) { return a.T <= 768 && a.dx != a.s && a.dx != a.dy; }

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s) {
    const Plan p = norm_plan(a.T, a.H);
    if (p.lanes == 16) {
        if (p.c == 1) run_norm<16, 1>(a, p, s);
        else run_norm<16, 2>(a, p, s);
    } else {
        if (p.c == 1) run_norm<64, 1>(a, p, s);
        else run_norm<64, 2>(a, p, s);
    }
    return hipGetLastError();
}

size_t norm_bwd_ws_bytes(int T, int H) { return (size_t)bwd_plan(T, H).grid * H * sizeof(float); }

hipError_t launch_add_rmsnorm_backward(const NormBwdArgs& a, void* ws, hipStream_t s) {
    float* part = static_cast<float*>(ws);
    int parts = 0;
    if (a.T) {
        Plan p = bwd_plan(a.T, a.H);
        parts = p.grid;
        if (one_launch(a)) {
            p.block = p.lanes == 16 ? p.block : p.block < 512 ? 512 : (p.block + 127) / 128 * 128;
            if (p.lanes == 16) {
                if (p.c == 1) run_norm_bwd<16, 1, true>(a, p, part, s);
                else run_norm_bwd<16, 2, true>(a, p, part, s);
            } else {
                if (p.c == 1) run_norm_bwd<64, 1, true>(a, p, part, s);
                else run_norm_bwd<64, 2, true>(a, p, part, s);
            }
            return hipGetLastError();
        }
        if (p.lanes == 16) {
            if (p.c == 1) run_norm_bwd<16, 1, false>(a, p, part, s);
            else run_norm_bwd<16, 2, false>(a, p, part, s);
        } else {
            if (p.c == 1) run_norm_bwd<64, 1, false>(a, p, part, s);
            else run_norm_bwd<64, 2, false>(a, p, part, s);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(norm_dw_kernel, dim3((a.H + 31) / 32), dim3(1024), 0, s, part, parts, a.H, a.dw);
    return hipGetLastError();
}

}  // namespace moe
