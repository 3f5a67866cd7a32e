// Per-expert counts of a routed batch, its balance loss and the gradient of
// the router's logits.
//
// With c_e the (token, slot) pairs of expert e, C their sum, f_e = c_e / C,
// p_t the softmax of token t's logits and S_e the sum of p_te over the valid
// tokens:
//   loss  = coef E k / C * sum_e f_e S_e
//   dl_te = coef E k / C * p_te (f_e - sum_j f_j p_tj)
// and, with the gradient dg of the gates g (a softmax over the chosen
// experts), dl_t,idx_j += g_j (dg_j - sum_i g_i dg_i).
//
// As the probabilities of a token sum to 1, f may be replaced by f' = f - 1/E
// in the gradient and the loss is coef E k / C * sum_t (sum_e f'_e p_te + 1/E).
// f' is formed from the integers c_e E - C, so nothing cancels in fp32 when the
// load is near even, and at an even load the gradient is 0 exactly.
//
// One wave (or 16 lanes, for few experts) takes one token after another and
// holds its logits in registers: a pass reads each logit once and writes each
// gradient once.  Its sums of p stay in registers too; a workgroup adds its
// waves' sums in a fixed order and writes one partial row, and a second kernel
// adds those.
#include "kernels.h"
#include "rows.h"

namespace moe {

// ------------------------------------------------------------------ counts

__global__ __launch_bounds__(256) void count_clear_kernel(uint32_t* __restrict__ counts, int E) {
    const int e = blockIdx.x * 256 + threadIdx.x;
    if (e < E) counts[e] = 0;
}

// Pairs [first, first + step) of each workgroup, counted in LDS and then added
// to `counts` (one workgroup and kWrite: written).  Integer additions: the
// order does not matter.  Ids outside [0, E) are not counted.
template <bool kWrite>
__global__ __launch_bounds__(1024) void count_kernel(const int32_t* __restrict__ idx, int64_t pairs, int k, int E,
                                                     const uint8_t* __restrict__ valid, uint32_t* __restrict__ counts) {
    __shared__ uint32_t bins[1024];
    for (int e = threadIdx.x; e < E; e += 1024) bins[e] = 0;
    __syncthreads();
    for (int64_t p = (int64_t)blockIdx.x * 1024 + threadIdx.x; p < pairs; p += (int64_t)gridDim.x * 1024) {
        if (valid && !valid[p / k]) continue;
        const uint32_t e = (uint32_t)idx[p];
        if (e < (uint32_t)E) atomicAdd(&bins[e], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 1024) {
        if (kWrite) counts[e] = bins[e];
        else if (bins[e]) atomicAdd(&counts[e], bins[e]);
    }
}

// ------------------------------------------------------------------ loss and gradient

// e^x for x <= 0: 2^t with t = x log2(e) rounded to fp32, corrected by the
// rounding's error (an fma gives it exactly) and by the part of log2(e) below
// fp32; within 2 units in the last place where a bare 2^t is off by |x| / 2.
// Gives 0 below about -87 and NaN for NaN.
__device__ __forceinline__ float exp_neg(float x) {
    const float kL = 1.44269502f, kLlo = 1.92596299e-8f;  // log2(e) = kL + kLlo
    const float t = x * kL;
    const float p = __builtin_amdgcn_exp2f(t);
    const float c = fmaf(x, kLlo, fmaf(x, kL, -t));
    return x < -104.0f ? 0.0f : fmaf(p * c, 0.693147182f, p);
}

// Sum and maximum over the kL lanes that hold a token.
template <int kL>
__device__ __forceinline__ float lanes_sum(float v) {
    return kL == 64 ? wave_sum_f32(v) : sum16_f32(v);
}
template <int kL>
__device__ __forceinline__ float lanes_max(float v) {
    v = fmaxf(v, dpp_f32<0xB1>(v));
    v = fmaxf(v, dpp_f32<0x4E>(v));
    v = fmaxf(v, dpp_f32<0x141>(v));
    v = fmaxf(v, dpp_f32<0x140>(v));
    if (kL == 16) return v;
    return fmaxf(fmaxf(readlane_f32(v, 0), readlane_f32(v, 16)), fmaxf(readlane_f32(v, 32), readlane_f32(v, 48)));
}

// kV neighbouring values of a row (kV = 4: one aligned load), and their store.
template <int kV>
__device__ __forceinline__ void load_v(const void* p, int64_t i, int f32, float* v) {
    if constexpr (kV == 4) {
        if (f32) {
            const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
            v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
            v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xFFFF0000u);
            v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xFFFF0000u);
        }
    } else {
        v[0] = f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
    }
}
template <int kV>
__device__ __forceinline__ void store_v(void* p, int64_t i, int f32, const float* v) {
    if constexpr (kV == 4) {
        if (f32) *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
        if (f32) static_cast<float*>(p)[i] = v[0];
        else static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_bits(v[0]);
    }
}

constexpr int kBalWaves = 8;

// Workspace: partial sums of p [workgroups][E] fp32, then per workgroup the
// sum of f' p over its tokens (fp64) and the number of tokens that count.
struct BalancePart {
    double fp;
    int64_t rows;
};

// Adds v to row[id]; the row is LDS of the token's own lanes.  Slots that name
// the same expert add in the order of the slots.
template <int kL>
__device__ __forceinline__ void add_slots(float* row, int slot, int k, int id, float v) {
    // a lane's claim is its slot's number, and a lane that does not find its own
    // there shares its expert
    const bool have = slot < k && id >= 0;
    if (have) row[id] = (float)slot;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const bool shared = have && row[id] != (float)slot;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const bool any = __any(shared);
    if (have) row[id] = any ? 0.0f : v;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (any) {
        for (int j = 0; j < k; ++j) {
            if (have && slot == j) row[id] += v;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }
}

template <int kL, int kV, int kI>
__global__ __launch_bounds__(64 * kBalWaves) void balance_kernel(BalanceArgs a, float* __restrict__ part, BalancePart* __restrict__ tail) {
    extern __shared__ __align__(16) float lds[];  // gates: one row of E values (rounded up to 4) per token in work; at the end the sums of p
    __shared__ unsigned long long total_s[kBalWaves];
    __shared__ double fp_s[kBalWaves * 64 / kL];
    __shared__ int64_t rows_s[kBalWaves * 64 / kL];
    constexpr int kTeams = kBalWaves * 64 / kL;  // tokens in work at a time
    const int t = threadIdx.x, l = t % kL, team = t / kL;
    const int E = a.E;

    unsigned long long total = 0;
    for (int e = t; e < E; e += 64 * kBalWaves) total += a.counts[e];
#pragma unroll
    for (int m = 1; m < 64; m *= 2) total += __shfl_xor(total, m, kWave);
    if (t % 64 == 0) total_s[t / 64] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kBalWaves; ++w) total += total_s[w];

    float f[kI][kV], sum[kI][kV];
    const double inv = total ? 1.0 / ((double)total * E) : 0.0;
    const float scale = total ? (float)((double)a.coef * E * a.k / (double)total) : 0.0f;
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int e = kV * (kL * i + l) + j;
            f[i][j] = e < E ? (float)((double)((int64_t)a.counts[e] * E - (int64_t)total) * inv) : 0.0f;
            sum[i][j] = 0.0f;
        }
    const int pitch = (E + 3) / 4 * 4;
    float* row_lds = lds + team * pitch;
    if (a.dgate) {
        for (int e = l; e < pitch; e += kL) row_lds[e] = 0.0f;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }

    double fp = 0.0;
    int64_t rows = 0;
    const int64_t step = (int64_t)gridDim.x * kTeams;
    // every team of a wave makes the same number of rounds
    for (int64_t first = (int64_t)blockIdx.x * kTeams + t / 64 * (64 / kL); first < a.T; first += step) {
        const int64_t row = first + (kL == 64 ? 0 : t % 64 / kL);
        const bool live = row < a.T;
        const bool on = live && (!a.valid || a.valid[row]);
        float v[kI][kV];
        float m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const int e = kV * (kL * i + l);
            if (on && e < E) {
                load_v<kV>(a.logits, row * a.ld + e, a.in_f32, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < kV; ++j) v[i][j] = -__builtin_inff();
            }
#pragma unroll
            for (int j = 0; j < kV; ++j) m = fmaxf(m, v[i][j]);
        }
        m = lanes_max<kL>(m);
        // no expert left (and nothing that is not a number): the token counts for nothing
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                // v = m = -inf would give NaN; a NaN stays one
                v[i][j] = v[i][j] == -__builtin_inff() ? 0.0f : exp_neg(v[i][j] - m);
                z += v[i][j];
            }
        z = lanes_sum<kL>(z);
        const bool empty = z == 0.0f;
        const float rz = empty ? 0.0f : __fdiv_rn(1.0f, z);
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                v[i][j] *= rz;
                sum[i][j] += v[i][j];
                q = fmaf(f[i][j], v[i][j], q);
            }
        q = lanes_sum<kL>(q);
        if (!empty) {
            fp += (double)q;
            rows += 1;
        }
        if (!a.dlogits) continue;
        int id = -1;
        if (a.dgate) {
            const bool slot = on && l < a.k;
            float g = 0.0f, dg = 0.0f;
            if (slot) {
                const int64_t p = row * a.k + l;
                id = a.idx[p];
                if ((uint32_t)id >= (uint32_t)E) id = -1;
                g = a.gate[p];
                dg = a.dgate[p];
            }
            const float mean = lanes_sum<kL>(g * dg);
            add_slots<kL>(row_lds, l, a.k, id, g * (dg - mean));
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < kI; ++i) {
                const int e = kV * (kL * i + l);
                if (e < E) {
                    float d[kV];
#pragma unroll
                    for (int j = 0; j < kV; ++j) {
                        d[j] = scale * v[i][j] * (f[i][j] - q);
                        if (a.dgate) d[j] += row_lds[e + j];
                    }
                    store_v<kV>(a.dlogits, row * a.ldd + e, a.out_f32, d);
                }
            }
        }
        if (a.dgate) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (id >= 0) row_lds[id] = 0.0f;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }

    // the workgroup's sums, team after team
    if (l == 0) {
        fp_s[team] = fp;
        rows_s[team] = rows;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int e = kV * (kL * i + l) + j;
            if (e < E) row_lds[e] = sum[i][j];
        }
    __syncthreads();
    for (int e = t; e < E; e += 64 * kBalWaves) {
        float s = 0.0f;
        for (int w = 0; w < kTeams; ++w) s += lds[w * pitch + e];
        part[(size_t)blockIdx.x * E + e] = s;
    }
    if (t == 0) {
        BalancePart b = {0.0, 0};
        for (int w = 0; w < kTeams; ++w) {
            b.fp += fp_s[w];
            b.rows += rows_s[w];
        }
        tail[blockIdx.x] = b;
    }
}

// The partial sums of `parts` workgroups: 64 experts a workgroup, its 16 waves
// each every sixteenth row, then the waves in turn; workgroup 0 adds the loss.
__global__ __launch_bounds__(1024) void balance_sum_kernel(const float* __restrict__ part, const BalancePart* __restrict__ tail,
                                                           int parts, int E, int k, float coef, const uint32_t* __restrict__ counts,
                                                           float* __restrict__ prob_sum, float* __restrict__ loss) {
    __shared__ float red[16][64];
    __shared__ double fp_s[16];
    __shared__ double rows_s[16];
    __shared__ double total_s[16];
    const int t = threadIdx.x, lane = t % 64, w = t / 64;
    const int e = blockIdx.x * 64 + lane;
    if (prob_sum) {
        float v = 0.0f;
        if (e < E)
            for (int p = w; p < parts; p += 16) v += part[(size_t)p * E + e];
        red[w][lane] = v;
    }
    if (blockIdx.x == 0) {
        double fp = 0.0, rows = 0.0, total = 0.0;
        for (int p = t; p < parts; p += 1024) {
            fp += tail[p].fp;
            rows += (double)tail[p].rows;
        }
        for (int i = t; i < E; i += 1024) total += (double)counts[i];
        fp = wave_sum_f64(fp);
        rows = wave_sum_f64(rows);
        total = wave_sum_f64(total);
        if (lane == 0) {
            fp_s[w] = fp;
            rows_s[w] = rows;
            total_s[w] = total;
        }
    }
    __syncthreads();
    if (prob_sum && w == 0 && e < E) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += red[i][lane];
        prob_sum[e] = s;
    }
    if (blockIdx.x == 0 && t == 0) {
        double fp = 0.0, rows = 0.0, total = 0.0;
        for (int i = 0; i < 16; ++i) {
            fp += fp_s[i];
            rows += rows_s[i];
            total += total_s[i];
        }
        loss[0] = total > 0.0 ? (float)((double)coef * E * k / total * (fp + rows / E)) : 0.0f;
    }
}

namespace {

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

int bal_lanes(int E, int k) { return E <= 64 && k <= 16 ? 16 : 64; }

int bal_grid(int T, int E, int k) {
    const int teams = kBalWaves * 64 / bal_lanes(E, k);
    const int need = (int)(((int64_t)T + teams - 1) / teams);
    return need < 1024 ? need : 1024;
}

template <int kL, int kV, int kI>
hipError_t run_balance(const BalanceArgs& a, float* part, BalancePart* tail, int grid, hipStream_t s) {
    const size_t lds = (size_t)(kBalWaves * 64 / kL) * ((a.E + 3) / 4 * 4) * sizeof(float);
    hipLaunchKernelGGL((balance_kernel<kL, kV, kI>), dim3(grid), dim3(64 * kBalWaves), lds, s, a, part, tail);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_counts(const int32_t* idx, int T, int k, int E, const uint8_t* valid, int accumulate, uint32_t* counts,
                                hipStream_t s) {
    const int64_t pairs = (int64_t)T * k;
    const int64_t need = (pairs + 4095) / 4096;
    if (need <= 1) {
        if (accumulate)
            hipLaunchKernelGGL((count_kernel<false>), dim3(1), dim3(1024), 0, s, idx, pairs, k, E, valid, counts);
        else
            hipLaunchKernelGGL((count_kernel<true>), dim3(1), dim3(1024), 0, s, idx, pairs, k, E, valid, counts);
        return hipGetLastError();
    }
    if (!accumulate) {
        hipLaunchKernelGGL(count_clear_kernel, dim3((E + 255) / 256), dim3(256), 0, s, counts, E);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int grid = (int)(need < 256 ? need : 256);
    hipLaunchKernelGGL((count_kernel<false>), dim3(grid), dim3(1024), 0, s, idx, pairs, k, E, valid, counts);
    return hipGetLastError();
}

size_t balance_ws_bytes(int T, int k, int E) {
    const int grid = bal_grid(T, E, k);
    return align16((size_t)grid * E * sizeof(float)) + (size_t)grid * sizeof(BalancePart);
}

hipError_t launch_balance_loss(const BalanceArgs& a, float* loss, float* prob_sum, void* ws, hipStream_t s) {
    const int grid = a.T ? bal_grid(a.T, a.E, a.k) : 0;
    float* part = static_cast<float*>(ws);
    BalancePart* tail = reinterpret_cast<BalancePart*>(static_cast<char*>(ws) + align16((size_t)grid * a.E * sizeof(float)));
    if (grid) {
        const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && (uintptr_t)a.logits % (a.in_f32 ? 16 : 8) == 0 &&
                         (!a.dlogits || (a.ldd % 4 == 0 && (uintptr_t)a.dlogits % (a.out_f32 ? 16 : 8) == 0));
        hipError_t e;
        if (bal_lanes(a.E, a.k) == 16)
            e = vec ? run_balance<16, 4, 1>(a, part, tail, grid, s) : run_balance<16, 1, 4>(a, part, tail, grid, s);
        else if (vec)
            e = a.E <= 256   ? run_balance<64, 4, 1>(a, part, tail, grid, s)
                : a.E <= 512 ? run_balance<64, 4, 2>(a, part, tail, grid, s)
                             : run_balance<64, 4, 4>(a, part, tail, grid, s);
        else
            e = a.E <= 128   ? run_balance<64, 1, 2>(a, part, tail, grid, s)
                : a.E <= 256 ? run_balance<64, 1, 4>(a, part, tail, grid, s)
                : a.E <= 512 ? run_balance<64, 1, 8>(a, part, tail, grid, s)
                             : run_balance<64, 1, 16>(a, part, tail, grid, s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(balance_sum_kernel, dim3((a.E + 63) / 64), dim3(1024), 0, s, part, tail, grid, a.E, a.k, a.coef, a.counts,
                       prob_sum, loss);
    return hipGetLastError();
}

}  // namespace moe
