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
// One wave (or 32 or 16 lanes, for few experts) takes one token after another and
// holds its logits in registers: a pass reads each logit once and writes each
// gradient once.  Its sums of p stay in registers too; a workgroup adds its
// waves' sums in a fixed order and writes one partial row, and a second kernel
// adds those.  Bound by memory, with the gradient's write as long as the read
// (32768 tokens of 512 experts with the gates' gradient: 30 us, 4.6 TB/s; the
// partial sums 4.5, the counts before it 4 and their clearing 1.4).
#include "kernels.h"
#include "rows.h"

namespace moe {

// ------------------------------------------------------------------ counts

__global__ __launch_bounds__(256) void count_clear_kernel(uint32_t* __restrict__ counts, int E) {
    const int e = blockIdx.x * 256 + threadIdx.x;
    if (e < E) counts[e] = 0;
}

// Pairs counted in LDS; ids outside [0, E) are not.  kOwn: a workgroup reads all
// pairs and counts a share of the experts, which it writes (or adds to).  Else it
// reads a share of the pairs and adds its counts of all experts to what others
// add (integers: the order does not matter).  Eight loads are on their way at a
// time; none stands in a branch, where it would be waited for (49152 pairs by
// one workgroup 22 us).
template <bool kOwn>
__global__ __launch_bounds__(1024) void count_kernel(const int32_t* __restrict__ idx, uint32_t pairs, uint32_t k, int E,
                                                     const uint8_t* __restrict__ valid, int accumulate, uint32_t* __restrict__ counts) {
    __shared__ uint32_t bins[1024];
    const int lo = kOwn ? (int)(E * blockIdx.x / gridDim.x) : 0, n = (kOwn ? (int)(E * (blockIdx.x + 1) / gridDim.x) : E) - lo;
    for (int e = threadIdx.x; e < n; e += 1024) bins[e] = 0;
    __syncthreads();
    const uint32_t step = kOwn ? 1024u : gridDim.x * 1024u, start = (kOwn ? 0u : blockIdx.x * 1024u) + threadIdx.x;
    // the pair's token and slot go along, which spares a division a pair
    const uint32_t tokens = pairs / k, dtok = step / k, dslot = step % k;
    uint32_t tok = start / k, slot = start % k;
    for (uint32_t p0 = start; p0 < pairs; p0 += 8 * step) {  // (below 2^31 + 2^19)
        uint32_t e[8], on[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t p = p0 + i * step;
            e[i] = (uint32_t)idx[p < pairs ? p : pairs - 1];
            if (valid) {
                on[i] = valid[tok < tokens ? tok : tokens - 1];
                tok += dtok;
                slot += dslot;
                if (slot >= k) {
                    slot -= k;
                    ++tok;
                }
            } else {
                on[i] = 1u;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = on[i] && p0 + i * step < pairs ? e[i] - (uint32_t)lo : ~0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e[i] < (uint32_t)n) atomicAdd(&bins[e[i]], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += 1024) {
        // (also where this workgroup alone has the expert: another stream's call may add to it)
        if (kOwn && !accumulate) counts[lo + e] = bins[e];
        else if (bins[e]) atomicAdd(&counts[lo + e], bins[e]);
    }
}

// ------------------------------------------------------------------ loss and gradient

// Sum and maximum over the kL lanes that hold a token.
template <int kL>
__device__ __forceinline__ float lanes_sum(float v) {
    if (kL == 64) return wave_sum_f32(v);
    v = sum16_f32(v);
    if (kL == 16) return v;
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
template <int kL>
__device__ __forceinline__ float lanes_max(float v) {
    v = fmaxf(v, dpp_f32<0xB1>(v));
    v = fmaxf(v, dpp_f32<0x4E>(v));
    v = fmaxf(v, dpp_f32<0x141>(v));
    v = fmaxf(v, dpp_f32<0x140>(v));
    if (kL == 16) return v;
    if (kL == 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    }
    return fmaxf(fmaxf(readlane_f32(v, 0), readlane_f32(v, 16)), fmaxf(readlane_f32(v, 32), readlane_f32(v, 48)));
}

// kV neighbouring values of a row (kV = 4: one aligned load), and their store
// (non-temporal: a gradient of 64 MB is not read back from L2; 41.1 -> 39.5 us
// for 32768 tokens of 512 experts).
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
        if (f32)
            __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i));
        else
            __builtin_nontemporal_store(u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])},
                                        reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p) + i));
    } else {
        if (f32) static_cast<float*>(p)[i] = v[0];
        else static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_bits(v[0]);
    }
}

constexpr int kBalWaves = 8;

// Workspace: partial sums of p [workgroups][E rounded up to 4] fp32, then per
// workgroup the sum of f' p over its tokens and the number of tokens that count.
struct BalancePart {
    double fp;
    double rows;
};
__host__ __device__ __forceinline__ int bal_pitch(int E) { return (E + 3) / 4 * 4; }

__device__ __forceinline__ void lds_settled() {  // LDS writes of a wave are seen by its later reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// row[id] = the sum of v over the token's slots that name id; row is LDS of the
// token's own lanes, and slots that name the same expert add in their order.
__device__ __forceinline__ void add_slots(float* row, int slot, int k, int id, float v) {
    // a lane's claim is its slot's number, and a lane that does not find its own
    // there shares its expert
    const bool have = id >= 0;
    if (have) row[id] = (float)slot;
    lds_settled();
    const bool any = __any(have && row[id] != (float)slot);
    lds_settled();
    if (have) row[id] = any ? 0.0f : v;
    lds_settled();
    if (any) {
        for (int j = 0; j < k; ++j) {
            if (have && slot == j) row[id] += v;
            lds_settled();
        }
    }
}

__device__ __forceinline__ float balance_value(double fp, double rows, double total, int E, int k, float coef) {
    return total > 0.0 ? (float)((double)coef * E * k / total * (fp + rows / E)) : 0.0f;
}

// kGates: the gates' gradient is taken in.  prob_sum and loss are written here
// when there is one workgroup, else the partial sums.
template <int kL, int kV, int kI, bool kGates>
__global__ __launch_bounds__(64 * kBalWaves) void balance_kernel(BalanceArgs a, float* __restrict__ part, BalancePart* __restrict__ tail,
                                                                 float* __restrict__ prob_sum, float* __restrict__ loss) {
    extern __shared__ __align__(16) float lds[];  // a row of E values (rounded up to 4) for each token in work
    constexpr int kTeams = kBalWaves * 64 / kL;   // tokens in work at a time
    __shared__ unsigned long long total_s[kBalWaves];
    __shared__ double fp_s[kTeams], rows_s[kTeams];
    const int t = threadIdx.x, l = t % kL, team = t / kL;
    const int E = a.E, pitch = bal_pitch(E);
    float* row_lds = lds + team * pitch;

    struct Token {
        float v[kI][kV];
        int id;
        float g, dg;
        bool on;
    };
    auto fetch = [&](int64_t row, Token& f) {
        f.on = row < a.T && (!a.valid || a.valid[row]);
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const int e = kV * (kL * i + l);
#pragma unroll
            for (int j = 0; j < kV; ++j) f.v[i][j] = -__builtin_inff();
            if (f.on && e < E) load_v<kV>(a.logits, row * a.ld + e, a.in_f32, f.v[i]);
        }
        f.id = -1;
        f.g = f.dg = 0.0f;
        if (kGates && f.on && l < a.k) {
            const int64_t p = row * a.k + l;
            f.id = a.idx[p];
            f.g = a.gate[p];
            f.dg = a.dgate[p];
        }
    };
    const int64_t step = (int64_t)gridDim.x * kTeams;
    int64_t first = (int64_t)blockIdx.x * kTeams + t / 64 * (64 / kL);  // of the wave: its teams make the same rounds
    const int off = kL == 64 ? 0 : t % 64 / kL;
    Token next;
    fetch(first + off, next);

    unsigned long long total = 0;
    for (int e = t; e < E; e += 64 * kBalWaves) total += a.counts[e];
#pragma unroll
    for (int m = 1; m < 64; m *= 2) total += __shfl_xor(total, m, kWave);
    if (t % 64 == 0) total_s[t / 64] = total;
    if (kGates)
        for (int e = l; e < pitch; e += kL) row_lds[e] = 0.0f;
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

    double fp = 0.0;
    int rows = 0;
    for (; first < a.T; first += step) {
        const int64_t row = first + off;
        Token f0 = next;
        if (first + step < a.T) fetch(row + step, next);
        auto& v = f0.v;
        float m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kV; ++j) m = fmaxf(m, v[i][j]);
        m = lanes_max<kL>(m);
        if (m == -__builtin_inff()) m = 0.0f;  // no expert left: every exponential is 0 (NaN stay what they are)
        float z = 0.0f, q = 0.0f;
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                v[i][j] = __builtin_amdgcn_exp2f((v[i][j] - m) * 1.44269504f);  // (m log2 e by itself might overflow)
                z += v[i][j];
                q = fmaf(f[i][j], v[i][j], q);
            }
        z = lanes_sum<kL>(z);
        q = lanes_sum<kL>(q);
        const bool empty = z == 0.0f;
        const float rz = empty ? 0.0f : __fdiv_rn(1.0f, z);
        q *= rz;
        if (!empty) {
            fp += (double)q;
            rows += 1;
        }
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                v[i][j] *= rz;
                sum[i][j] += v[i][j];
            }
        if (!a.dlogits) continue;
        if (kGates) {
            if ((uint32_t)f0.id >= (uint32_t)E) f0.id = -1;
            add_slots(row_lds, l, a.k, f0.id, f0.g * (f0.dg - lanes_sum<kL>(f0.g * f0.dg)));
        }
        if (row < a.T) {
            const float sq = scale * q;
#pragma unroll
            for (int i = 0; i < kI; ++i) {
                const int e = kV * (kL * i + l);
                if (e < E) {
                    float d[kV];
#pragma unroll
                    for (int j = 0; j < kV; ++j) d[j] = fmaf(v[i][j], fmaf(scale, f[i][j], -sq), kGates ? row_lds[e + j] : 0.0f);
                    store_v<kV>(a.dlogits, row * a.ldd + e, a.out_f32, d);
                }
            }
        }
        if (kGates) {
            lds_settled();
            if (f0.id >= 0) row_lds[f0.id] = 0.0f;
            lds_settled();
        }
    }

    // the workgroup's sums, team after team
    if (l == 0) {
        fp_s[team] = fp;
        rows_s[team] = rows;
    }
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int e = kV * (kL * i + l) + j;
            if (e < pitch) row_lds[e] = sum[i][j];
        }
    __syncthreads();
    const bool alone = gridDim.x == 1;
    for (int e = t; e < pitch; e += 64 * kBalWaves) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kTeams; ++w) s += lds[w * pitch + e];
        if (!alone) part[(size_t)blockIdx.x * pitch + e] = s;
        else if (prob_sum && e < E) prob_sum[e] = s;
    }
    if (t == 0) {
        BalancePart b = {0.0, 0.0};
        for (int w = 0; w < kTeams; ++w) {
            b.fp += fp_s[w];
            b.rows += rows_s[w];
        }
        if (!alone) tail[blockIdx.x] = b;
        else loss[0] = balance_value(b.fp, b.rows, (double)total, E, a.k, a.coef);
    }
}

// The partial sums of `parts` workgroups, in a fixed order: 32 experts (whole
// lines) a workgroup; thread (p, q) adds rows p, p + 128, .. of experts 4q..4q+3,
// eight loads on their way at a time, then the 128 sums are added in order of p
// modulo 16.  Workgroup 0 adds the loss.
__global__ __launch_bounds__(1024) void balance_sum_kernel(const float* __restrict__ part, const BalancePart* __restrict__ tail,
                                                           int parts, int E, int k, float coef, const uint32_t* __restrict__ counts,
                                                           float* __restrict__ prob_sum, float* __restrict__ loss) {
    __shared__ __align__(16) f32x4_t red[128][8];
    __shared__ double fp_s[16], rows_s[16], total_s[16];
    const int t = threadIdx.x, lane = t % 64, w = t / 64;
    const int q = t % 8, p0 = t / 8, pitch = bal_pitch(E), e = blockIdx.x * 32 + 4 * q;
    f32x4_t v = f32x4_t(0.0f);
    if (prob_sum && e < pitch) v = sum_rows(part + e, parts, pitch, p0);
    red[p0][q] = v;
    if (blockIdx.x == 0) {
        double fp = 0.0, rows = 0.0, total = 0.0;
        for (int p = t; p < parts; p += 1024) {
            fp += tail[p].fp;
            rows += tail[p].rows;
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
    v = sum_128(v, red, p0, q);
    if (prob_sum && p0 == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e + j < E) prob_sum[e + j] = v[j];
    }
    if (blockIdx.x == 0 && t == 0) {
        double fp = 0.0, rows = 0.0, total = 0.0;
        for (int i = 0; i < 16; ++i) {
            fp += fp_s[i];
            rows += rows_s[i];
            total += total_s[i];
        }
        loss[0] = balance_value(fp, rows, total, E, k, coef);
    }
}

namespace {

// Up to here one launch counts.  It spares the host 2.5 us a call, but each of its workgroups reads all pairs; the two
// launches take 4.0 to 4.8 us in a graph whatever the number.  One launch against two, 61 or 512 experts, us a call: 20000
// pairs 5.5, 7.9; 49146 7.0, 7.9; 65000 8.5, 7.9 (in a graph 10000 3.9, 4.4; 20000 4.6, 4.3; 49146 7.2, 4.4; 65000 8.7, 4.4).
// So the border is that of calls outside a graph, which pay for it inside one from about 15000 pairs on.  Below 16 experts
// there is one workgroup, the slower form from about 28000 pairs on (8 experts: 20000 6.1, 7.8; 49150 11.4, 7.9).
constexpr uint32_t kCountOwn = 49152;

// Lanes of a token: the sums over them cost as much for few experts as for many, and short rows share a wave (65536
// tokens of 128 experts: 64 lanes 35 us, 32 27.8; of 256, bf16: 35.3, 33.2; 300 of 256: 10.8, 11.7; 512 experts gain
// nothing).
int bal_lanes(int E, int k) { return E <= 64 && k <= 16 ? 16 : E <= 256 && k <= 32 ? 32 : 64; }

// A few rounds of one workgroup cost less than the sums' kernel.  More workgroups keep more loads on their way and write
// more partial rows (65536 tokens of 256, bf16: 256 workgroups 55 us, 512 41, 768 35, 1024 35; 32768 of 512: 39, 40, 39, 40;
// 16384 of 1024: 40, 41, 44, 45).
int bal_grid(int T, int E, int k) {
    const int teams = kBalWaves * 64 / bal_lanes(E, k), most = E > 512 ? 256 : 768;
    const int need = (int)(((int64_t)T + teams - 1) / teams);
    return need <= 4 ? 1 : need < most ? need : most;
}

template <int kL, int kV, int kI>
hipError_t run_balance(const BalanceArgs& a, float* part, BalancePart* tail, float* prob_sum, float* loss, int grid, hipStream_t s) {
    const size_t lds = (size_t)(kBalWaves * 64 / kL) * bal_pitch(a.E) * sizeof(float);
    const dim3 g(grid), b(64 * kBalWaves);
    if (a.dgate) hipLaunchKernelGGL((balance_kernel<kL, kV, kI, true>), g, b, lds, s, a, part, tail, prob_sum, loss);
    else hipLaunchKernelGGL((balance_kernel<kL, kV, kI, false>), g, b, lds, s, a, part, tail, prob_sum, loss);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_counts(const int32_t* idx, int T, int k, int E, const uint8_t* valid, int accumulate, uint32_t* counts,
                                hipStream_t s) {
    const uint32_t pairs = (uint32_t)T * (uint32_t)k;  // (fits 31 bits)
    if (pairs <= kCountOwn) {
        const dim3 grid(pairs <= 1024 || E < 16 ? 1 : 16), block(1024);
        hipLaunchKernelGGL((count_kernel<true>), grid, block, 0, s, idx, pairs, (uint32_t)k, E, valid, accumulate, counts);
        return hipGetLastError();
    }
    if (!accumulate) {
        hipLaunchKernelGGL(count_clear_kernel, dim3((E + 255) / 256), dim3(256), 0, s, counts, E);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const uint32_t need = (pairs + 4095) / 4096;  // (more than 64 meet at the same counters)
    hipLaunchKernelGGL((count_kernel<false>), dim3(need < 64 ? need : 64), dim3(1024), 0, s, idx, pairs, (uint32_t)k, E, valid, 1,
                       counts);
    return hipGetLastError();
}

size_t balance_ws_bytes(int T, int k, int E) {
    const int grid = bal_grid(T, E, k);
    return (size_t)grid * (bal_pitch(E) * sizeof(float) + sizeof(BalancePart));
}

hipError_t launch_balance_loss(const BalanceArgs& a, float* loss, float* prob_sum, void* ws, hipStream_t s) {
    const int grid = a.T ? bal_grid(a.T, a.E, a.k) : 0;
    float* part = static_cast<float*>(ws);
    BalancePart* tail = reinterpret_cast<BalancePart*>(part + (size_t)grid * bal_pitch(a.E));
    if (grid) {
        const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && (uintptr_t)a.logits % (a.in_f32 ? 16 : 8) == 0 &&
                         (!a.dlogits || (a.ldd % 4 == 0 && (uintptr_t)a.dlogits % (a.out_f32 ? 16 : 8) == 0));
        hipError_t e;
#define MOE_BALANCE(kL, kV, kI) run_balance<kL, kV, kI>(a, part, tail, prob_sum, loss, grid, s)
        if (bal_lanes(a.E, a.k) == 16)
            e = vec ? MOE_BALANCE(16, 4, 1) : MOE_BALANCE(16, 1, 4);
        else if (bal_lanes(a.E, a.k) == 32)
            e = vec ? a.E <= 128 ? MOE_BALANCE(32, 4, 1) : MOE_BALANCE(32, 4, 2) : a.E <= 128 ? MOE_BALANCE(32, 1, 4) : MOE_BALANCE(32, 1, 8);
        else if (vec)
            e = a.E <= 256 ? MOE_BALANCE(64, 4, 1) : a.E <= 512 ? MOE_BALANCE(64, 4, 2) : MOE_BALANCE(64, 4, 4);
        else
            e = a.E <= 128   ? MOE_BALANCE(64, 1, 2)
                : a.E <= 256 ? MOE_BALANCE(64, 1, 4)
                : a.E <= 512 ? MOE_BALANCE(64, 1, 8)
                             : MOE_BALANCE(64, 1, 16);
#undef MOE_BALANCE
        if (e != hipSuccess || grid == 1) return e;
    }
    hipLaunchKernelGGL(balance_sum_kernel, dim3((a.E + 31) / 32), dim3(1024), 0, s, part, tail, grid, a.E, a.k, a.coef, a.counts,
                       prob_sum, loss);
    return hipGetLastError();
}

}  // namespace moe
