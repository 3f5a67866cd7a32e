// The whole MoE layer for at most 16 tokens in two kernels (moe_layer_few).
//
//   y_t = sum_j gate_tj down_e( silu(gate_e x_t) * (up_e x_t) )  +  s_t shared(x_t)
//
// Few tokens read every touched expert once and use each weight for one or
// two rows, so the bytes bound the call, and at one token the launches and
// waits between its dependent steps.  Hence two launches and as few waits:
//
//  few_front_kernel: the router's logits (exact, fp64 sums rounded once) and,
//    independent of them, gate/up of the shared expert; also clears the second
//    kernel's counters.
//  few_experts_kernel: every workgroup selects the top k of every token by
//    itself from the logits (cheaper than a third launch or a wait), then takes
//    a ticket.  The first tickets are gate/up workgroups: they stream gate and
//    up rows, write gate_tj * h (fp32) and count themselves done.  The others
//    own 8 outputs each: they load their first down rows, wait for the count,
//    and sum all experts and the shared one in fp32, in a fixed order.
//
// The wait always ends: a workgroup that waits holds a ticket that was given
// out after all gate/up tickets, so every gate/up workgroup is already running,
// and those wait for nothing.  (No workgroup needs another to be resident that
// is not, whatever else runs on the GPU.)  It is bounded all the same, for a
// workspace that a second call clears meanwhile: then y is NaN.
// h passes between compute dies, whose L2s are not coherent within a kernel:
// stores and loads of it go past them (agent scope, sc1), and a store has
// completed before its workgroup counts itself done.
//
// Weights stream in 16-byte pieces with the non-temporal hint; a piece is 8
// bf16, 16 E4M3 or 32 4-bit inputs of one column.
#include "fp8.h"
#include "ffn_internal.h"
#include "select.h"

namespace moe {

namespace {

constexpr int kFewThreads = 512, kFewWaves = kFewThreads / kWave;
constexpr int kFewCols = 8;        // outputs of a down workgroup
constexpr int kFewMaxPairs = kFewMaxT * 64;
constexpr int kAgent = 16;         // cache policy of buffer accesses: sc1

enum { F_BF16 = 0, F_FP8 = 1, F_AWQ = 2 };

struct FewProj {
    const void* w;          // bf16 [E][O][I], E4M3 codes [E][O][I], 4-bit codes [E][O][I/8]
    const float* bscales;   // E4M3: [E][O/128][I/128]
    const uint16_t* scales; // 4-bit: [E][I/32][O] fp16
    const int32_t* qzeros;  // 4-bit: [E][I/32][O/8]
};

struct FewArgs {
    const uint16_t* x;      // [T][H]
    const uint16_t* router; // [E][H]
    const float* shared_scale;
    FewProj gate, up, down, sgate, sup, sdown;
    int T, H, E, k, F, Fs;  // Fs = 0: no shared expert
    int gateup_wgs;
    uint32_t* counters;     // [0] tickets, [32 (1 + i)] done, i < 8
    float* logits;          // [T][E]
    float* hs;              // [T][Fs]
    float* h;               // [T k][F], rows grouped by expert
    uint16_t* y;            // [T][H]
    int32_t* topk_idx;      // [T][k] or nullptr
};

// Inputs of a 16-byte piece.
template <int FMT>
struct Piece {
    static constexpr int N = FMT == F_BF16 ? 8 : FMT == F_FP8 ? 16 : 32;
};

// One piece of a column and what scales it.
template <int FMT>
struct Weights {
    uint4 w;
    float s;        // E4M3: block scale; 4-bit: group scale
    float z;        // 4-bit: zero point
};

template <int FMT>
__device__ __forceinline__ void load_piece(Weights<FMT>& d, const FewProj& p, size_t e, int O, int I, int o, int c) {
    constexpr int N = Piece<FMT>::N;
    const size_t row = e * O + o;
    d.w = ld_stream(reinterpret_cast<const uint4*>(p.w) + row * (I / N) + c);
    if (FMT == F_FP8) d.s = p.bscales[(e * (O / 128) + o / 128) * (I / 128) + c / 8];
    if (FMT == F_AWQ) {
        const size_t grp = e * (I / 32) + c;
        d.s = f16_to_f32(p.scales[grp * O + o]);
        const int c8 = o & 7, nib = (c8 & 1) ? 4 + (c8 >> 1) : (c8 >> 1);  // AWQ order of zero words
        d.z = (float)(((uint32_t)p.qzeros[grp * (O / 8) + (o >> 3)] >> (4 * nib)) & 15u);
    }
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Dot of a piece with bf16 inputs x (N / 8 vectors of 8).
template <int FMT>
__device__ __forceinline__ float dot_x(const Weights<FMT>& d, const uint4 (&x)[Piece<FMT>::N / 8]) {
    float acc = 0.0f;
    if constexpr (FMT == F_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = dot2_bf16(word(d.w, i), word(x[0], i), acc);
        return acc;
    } else if constexpr (FMT == F_FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // E4M3 is exact in bf16
            const int w = (int)word(d.w, i);
            const uint32_t lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
            const uint32_t hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
            acc = dot2_bf16(lo, word(x[i / 2], 2 * (i & 1)), acc);
            acc = dot2_bf16(hi, word(x[i / 2], 2 * (i & 1) + 1), acc);
        }
        return acc * d.s;
    } else {
        // 128 + q is exact in bf16 (bits 0x4300 | q): s (sum (128 + q) x - (128 + z) sum x)
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = word(d.w, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // nibbles j and j + 4 with inputs j and j + 4
                const uint32_t q = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
                const uint32_t lo = word(x[i], j / 2), hi = word(x[i], 2 + j / 2);
                const uint32_t xx = (j & 1) ? __builtin_amdgcn_perm(hi, lo, 0x07060302u) : __builtin_amdgcn_perm(hi, lo, 0x05040100u);
                acc = dot2_bf16(q, xx, acc);
                sum = dot2_bf16(0x3F803F80u, xx, sum);
            }
        }
        return d.s * (acc - (128.0f + d.z) * sum);
    }
}

// Dot of a piece with fp32 inputs h.
template <int FMT>
__device__ __forceinline__ float dot_h(const Weights<FMT>& d, const f32x4_t (&h)[Piece<FMT>::N / 4]) {
    float acc = 0.0f;
    if constexpr (FMT == F_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = word(d.w, i);
            acc = fmaf(__uint_as_float(w << 16), h[i / 2][2 * (i & 1)], acc);
            acc = fmaf(__uint_as_float(w & 0xFFFF0000u), h[i / 2][2 * (i & 1) + 1], acc);
        }
        return acc;
    } else if constexpr (FMT == F_FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int w = (int)word(d.w, i);
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
            acc = fmaf(lo[0], h[i][0], acc);
            acc = fmaf(lo[1], h[i][1], acc);
            acc = fmaf(hi[0], h[i][2], acc);
            acc = fmaf(hi[1], h[i][3], acc);
        }
        return acc * d.s;
    } else {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = word(d.w, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = h[2 * i + j / 4][j & 3];
                acc = fmaf((float)((w >> (4 * j)) & 15u), v, acc);
                sum += v;
            }
        }
        return d.s * (acc - d.z * sum);
    }
}

// Sum over aligned groups of L lanes, in every lane of the group.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = L / 2; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
    return v;
}

__device__ __forceinline__ uint4 load_x8(const uint16_t* x, size_t row, int H, int i) {
    return *reinterpret_cast<const uint4*>(x + row * H + i);
}

// Gate and up of the columns of one pass of a wave (64 / L columns, L lanes
// each) for the tokens token(i), i < n: done(i, column, gate, up) is called in
// the group's lanes.  U pieces of gate and of up are loaded at a time; columns
// longer than U L pieces add their parts in `part` (LDS of the wave: 2 floats
// per token and column of the pass).
template <int FMT, int L, int U, class Tok, class Done>
__device__ __forceinline__ void gateup_pass(const FewProj& pg, const FewProj& pu, size_t e, int F, int H, int col,
                                            const uint16_t* x, int n, float* part, Tok token, Done done) {
    constexpr int N = Piece<FMT>::N, C = kWave / L;
    const int lane = threadIdx.x & 63, gl = lane % L, gi = lane / L;
    const int pieces = H / N, o = min(col + gi, F - 1);
    const bool one = pieces <= U * L;
    for (int c0 = 0; c0 < pieces; c0 += U * L) {
        Weights<FMT> wg[U], wu[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * L + gl;
            in[u] = c < pieces;
            load_piece<FMT>(wg[u], pg, e, F, H, o, min(c, pieces - 1));
            load_piece<FMT>(wu[u], pu, e, F, H, o, min(c, pieces - 1));
        }
        for (int i = 0; i < n; ++i) {
            const int t = token(i);
            float g = 0.0f, v = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = min(c0 + u * L + gl, pieces - 1);
                uint4 xv[N / 8];
#pragma unroll
                for (int q = 0; q < N / 8; ++q) xv[q] = load_x8(x, (size_t)t, H, c * N + 8 * q);
                const float a = dot_x<FMT>(wg[u], xv), b = dot_x<FMT>(wu[u], xv);
                g += in[u] ? a : 0.0f;
                v += in[u] ? b : 0.0f;
            }
            g = group_sum<L>(g);
            v = group_sum<L>(v);
            if (!one) {
                float* q = part + (i * C + gi) * 2;
                if (c0 > 0) {
                    g += q[0];
                    v += q[1];
                }
                if (gl == 0) {
                    q[0] = g;
                    q[1] = v;
                }
            }
            if (c0 + U * L >= pieces) done(i, col + gi, gl == 0 && col + gi < F, g, v);
        }
    }
}

// Lanes of a column: a column of 2560 inputs takes 5 pieces a lane.
template <int FMT>
struct GateUpShape {
    static constexpr int L = FMT == F_BF16 ? 64 : FMT == F_FP8 ? 32 : 16, C = kWave / L, U = 5;
};
// Down: 640 inputs take 5 pieces a lane (4-bit: 3).
template <int FMT>
struct DownShape {
    static constexpr int L = FMT == F_BF16 ? 16 : 8, C = kWave / L, U = FMT == F_AWQ ? 3 : 5;
};

// Logits of one expert for TT tokens: exact bf16 products summed in fp64.
template <int TT>
__device__ __forceinline__ void front_logits(const FewArgs& a, int e, int lane) {
    double acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.0;
    for (int c = lane * 8; c < a.H; c += kWave * 8) {
        const uint4 r = *reinterpret_cast<const uint4*>(a.router + (size_t)e * a.H + c);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const uint4 xv = load_x8(a.x, (size_t)min(t, a.T - 1), a.H, c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t w = word(r, i), v = word(xv, i);
                acc[t] = fma((double)__uint_as_float(w << 16), (double)__uint_as_float(v << 16), acc[t]);
                acc[t] = fma((double)__uint_as_float(w & 0xFFFF0000u), (double)__uint_as_float(v & 0xFFFF0000u), acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const double s = wave_sum_f64(acc[t]);
        if (lane == 0 && t < a.T) a.logits[(size_t)t * a.E + e] = (float)s;
    }
}

constexpr int kFrontThreads = 256, kFrontWaves = kFrontThreads / kWave;

// Wave w of the grid: logits of expert w, or columns of the shared expert.
template <int TT>
__global__ __launch_bounds__(kFrontThreads) void few_front_kernel(const FewArgs a) {
    __shared__ float part[kFrontWaves][kFewMaxT * 2];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    if (blockIdx.x == 0 && threadIdx.x < 9) a.counters[32 * threadIdx.x] = 0;
    const int w = blockIdx.x * kFrontWaves + wv;
    if (w < a.E) {
        front_logits<TT>(a, w, lane);
    } else if (w - a.E < a.Fs) {
        using S = GateUpShape<F_BF16>;
        gateup_pass<F_BF16, S::L, S::U>(
            a.sgate, a.sup, 0, a.Fs, a.H, w - a.E, a.x, a.T, part[wv], [](int i) { return i; },
            [&](int i, int col, bool mine, float g, float u) {
                if (mine) a.hs[(size_t)i * a.Fs + col] = silu(g) * u * (a.shared_scale ? a.shared_scale[i] : 1.0f);
            });
    }
}

struct FewLists {
    int32_t idx[kFewMaxPairs];    // expert of pair t k + j
    float gate[kFewMaxPairs];
    int32_t count[kFewMaxPairs];  // pairs of the expert, at its first pair; 0 elsewhere
    int32_t order[kFewMaxPairs];  // pairs grouped by expert
    int32_t first[kFewMaxPairs];  // expert slot: first row in `order`; its expert is that of the row's pair
    int32_t slots;
};

// Selection and grouping, the same in every workgroup: the top k of every
// token, then the pairs grouped by expert, experts in the order of their first
// pair, pairs ascending.  P is at most 16 * 64: every pair looks at all others.
__device__ __forceinline__ void few_select(const FewArgs& a, FewLists& s) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, P = a.T * a.k;
    for (int t = wv; t < a.T; t += kFewWaves) {
        if (a.E <= 512) select_token<8>(a.logits, (size_t)t, a.E, a.k, a.k, lane, s.idx, nullptr, s.gate);
        else select_token<16>(a.logits, (size_t)t, a.E, a.k, a.k, lane, s.idx, nullptr, s.gate);
    }
    if (threadIdx.x == 0) s.slots = 0;
    __syncthreads();
    int lead[kFewMaxPairs / kFewThreads], rank[kFewMaxPairs / kFewThreads];
#pragma unroll
    for (int r = 0; r < kFewMaxPairs / kFewThreads; ++r) {
        const int p = threadIdx.x + r * kFewThreads;
        lead[r] = rank[r] = 0;
        if (p >= P) continue;
        const int e = s.idx[p];
        int before = 0, all = 0, f = p;
        for (int q = 0; q < P; ++q) {
            const bool same = s.idx[q] == e;
            all += same;
            before += same && q < p;
            f = same && q < f ? q : f;
        }
        lead[r] = f;
        rank[r] = before;
        s.count[p] = before == 0 ? all : 0;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kFewMaxPairs / kFewThreads; ++r) {
        const int p = threadIdx.x + r * kFewThreads;
        if (p >= P) continue;
        int start = 0, slot = 0;
        for (int q = 0; q < lead[r]; ++q) {
            const int c = s.count[q];
            start += c;
            slot += c > 0;
        }
        s.order[start + rank[r]] = p;
        if (rank[r] == 0) {
            s.first[slot] = start;
            atomicAdd(&s.slots, 1);
        }
    }
    __syncthreads();
}

template <int FMT>
__global__ __launch_bounds__(kFewThreads, 4) void few_experts_kernel(const FewArgs a) {
    __shared__ FewLists s;
    __shared__ float acc[kFewWaves][kFewMaxT][kFewCols];   // down: sums; gate/up: parts of long columns
    __shared__ int s_ticket, s_ok;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int P = a.T * a.k;
    int ticket = 0;
    if (threadIdx.x == 0) ticket = (int)__hip_atomic_fetch_add(a.counters, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    few_select(a, s);
    if (threadIdx.x == 0) s_ticket = ticket;
    __syncthreads();
    ticket = s_ticket;
    const int slots = s.slots;
    const __amdgpu_buffer_rsrc_t rh = fp8_rsrc(a.h, (uint32_t)P * (uint32_t)a.F * 4u);
    auto slot_end = [&](int u) { return u + 1 < slots ? s.first[u + 1] : P; };

    if (ticket < a.gateup_wgs) {
        using S = GateUpShape<FMT>;
        // passes (expert slot, columns) in contiguous ranges over the waves
        const int per = (a.F + S::C - 1) / S::C, n = slots * per;
        const int nw = a.gateup_wgs * kFewWaves, w = ticket * kFewWaves + wv;
        const int q0 = (int)((int64_t)n * w / nw), q1 = (int)((int64_t)n * (w + 1) / nw);
        for (int q = q0; q < q1; ++q) {
            const int u = q / per, col = (q - u * per) * S::C;
            const int r0 = s.first[u], rows = slot_end(u) - r0;
            gateup_pass<FMT, S::L, S::U>(
                a.gate, a.up, (size_t)s.idx[s.order[r0]], a.F, a.H, col, a.x, rows, &acc[wv][0][0],
                [&](int i) { return s.order[r0 + i] / a.k; },
                [&](int i, int c, bool mine, float g, float v) {
                    const float h = silu(g) * v * s.gate[s.order[r0 + i]];
                    if (mine)
                        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(h), rh,
                                                              (int)(((uint32_t)(r0 + i) * (uint32_t)a.F + (uint32_t)c) * 4u), 0,
                                                              kAgent);
                });
        }
        if (ticket == 0 && a.topk_idx)
            for (int p = threadIdx.x; p < P; p += kFewThreads) a.topk_idx[p] = s.idx[p];
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the stores have completed
        __syncthreads();
        if (threadIdx.x == 0)
            __hip_atomic_fetch_add(a.counters + 32 * (1 + ticket % 8), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return;
    }

    // ---- down: outputs o0 .. o0 + 7, experts dealt over the waves
    using S = DownShape<FMT>;
    constexpr int N = Piece<FMT>::N;
    const int o0 = (ticket - a.gateup_wgs) * kFewCols;
    for (int i = threadIdx.x; i < kFewWaves * kFewMaxT * kFewCols; i += kFewThreads) (&acc[0][0][0])[i] = 0.0f;
    if (threadIdx.x == 0) s_ok = 1;
    __syncthreads();
    if (wv == 0) {
        // all gate/up workgroups done?  Lanes 0..7 read the eight counts.
        const uint64_t begin = wall_clock64();
        for (;;) {
            uint32_t c = 0;
            if (lane < 8) c = __hip_atomic_load(a.counters + 32 * (1 + lane), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int m = 4; m >= 1; m >>= 1) c += __shfl_xor(c, m, kWave);
            if ((uint32_t)__builtin_amdgcn_readfirstlane((int)c) >= (uint32_t)a.gateup_wgs) break;
            if (wall_clock64() - begin > 400000000ull) {  // 4 s of the 100 MHz counter
                if (lane == 0) s_ok = 0;
                break;
            }
            __builtin_amdgcn_s_sleep(2);
        }
    }
    __syncthreads();
    asm volatile("" ::: "memory");

    const int gl = lane % S::L, gi = lane / S::L;
    const int pieces = a.F / N;
    for (int u = wv; u < slots; u += kFewWaves) {
        const int r0 = s.first[u], rows = slot_end(u) - r0;
        const size_t e = (size_t)s.idx[s.order[r0]];
        for (int cb = 0; cb < kFewCols; cb += S::C) {
            const int o = min(o0 + cb + gi, a.H - 1);
            for (int c0 = 0; c0 < pieces; c0 += S::U * S::L) {
                Weights<FMT> w[S::U];
#pragma unroll
                for (int i = 0; i < S::U; ++i)
                    load_piece<FMT>(w[i], a.down, e, a.H, a.F, o, min(c0 + i * S::L + gl, pieces - 1));
                for (int r = 0; r < rows; ++r) {
                    float v = 0.0f;
#pragma unroll
                    for (int i = 0; i < S::U; ++i) {
                        const int c = c0 + i * S::L + gl;
                        f32x4_t h[N / 4];
#pragma unroll
                        for (int q = 0; q < N / 4; ++q)
                            h[q] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                rh, (int)(((uint32_t)(r0 + r) * (uint32_t)a.F + (uint32_t)(min(c, pieces - 1) * N + 4 * q)) * 4u),
                                0, kAgent));
                        const float d = dot_h<FMT>(w[i], h);
                        v += c < pieces ? d : 0.0f;
                    }
                    v = group_sum<S::L>(v);
                    if (gl == 0) acc[wv][s.order[r0 + r] / a.k][cb + gi] += v;
                }
            }
        }
    }
    if (a.Fs) {
        // the shared expert: tokens dealt over the waves
        using B = DownShape<F_BF16>;
        const int sl = lane % B::L, si = lane / B::L, sp = a.Fs / 8;
        for (int t = wv; t < a.T; t += kFewWaves)
            for (int cb = 0; cb < kFewCols; cb += B::C) {
                const int o = min(o0 + cb + si, a.H - 1);
                float v = 0.0f;
                for (int c = sl; c < sp; c += B::L) {
                    Weights<F_BF16> w;
                    load_piece<F_BF16>(w, a.sdown, 0, a.H, a.Fs, o, c);
                    const f32x4_t* hp = reinterpret_cast<const f32x4_t*>(a.hs + (size_t)t * a.Fs + 8 * c);
                    const f32x4_t h[2] = {hp[0], hp[1]};
                    v += dot_h<F_BF16>(w, h);
                }
                v = group_sum<B::L>(v);
                if (sl == 0) acc[wv][t][cb + si] += v;
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * kFewCols; i += kFewThreads) {
        const int t = i / kFewCols, c = i % kFewCols;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kFewWaves; ++q) v += acc[q][t][c];
        if (!s_ok) v = __uint_as_float(0x7FC00000u);
        if (o0 + c < a.H) a.y[(size_t)t * a.H + o0 + c] = (uint16_t)f32_to_bf16_bits(v);
    }
}

FewProj few_proj(const moe_proj& p) {
    FewProj d{};
    d.w = p.fmt == MOE_W_BF16 ? (const void*)p.w : p.fmt == MOE_W_FP8_BLOCK ? (const void*)p.codes : (const void*)p.qweight;
    d.bscales = p.block_scales;
    d.scales = p.scales;
    d.qzeros = p.qzeros;
    return d;
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace

bool few_supported(const moe_experts* ex, const moe_experts* sh) {
    const int f = ex->gate.fmt;
    return (f == MOE_W_BF16 || f == MOE_W_FP8_BLOCK || f == MOE_W_AWQ_G32_OM) && (!sh || sh->gate.fmt == MOE_W_BF16);
}

size_t few_ws_bytes(int T, int k, const moe_experts* ex, const moe_experts* sh) {
    return up256(9 * 32 * 4) + up256((size_t)T * ex->num_experts * 4) + up256(sh ? (size_t)T * sh->inter * 4 : 0) +
           up256((size_t)T * k * ex->inter * 4);
}

hipError_t launch_layer_few(const uint16_t* x, int T, const uint16_t* router, int k, const moe_experts* ex,
                            const moe_experts* sh, const float* shared_scale, uint16_t* y, int32_t* topk_idx, void* ws,
                            hipStream_t s) {
    FewArgs a{};
    a.x = x;
    a.router = router;
    a.shared_scale = shared_scale;
    a.gate = few_proj(ex->gate);
    a.up = few_proj(ex->up);
    a.down = few_proj(ex->down);
    a.T = T; a.H = ex->hidden; a.E = ex->num_experts; a.k = k; a.F = ex->inter;
    if (sh) {
        a.sgate = few_proj(sh->gate);
        a.sup = few_proj(sh->up);
        a.sdown = few_proj(sh->down);
        a.Fs = sh->inter;
    }
    char* w = static_cast<char*>(ws);
    a.counters = reinterpret_cast<uint32_t*>(w);
    w += up256(9 * 32 * 4);
    a.logits = reinterpret_cast<float*>(w);
    w += up256((size_t)T * a.E * 4);
    a.hs = reinterpret_cast<float*>(w);
    w += up256((size_t)T * a.Fs * 4);
    a.h = reinterpret_cast<float*>(w);
    a.y = y;
    a.topk_idx = topk_idx;
    a.gateup_wgs = 256;
    const dim3 front((a.E + a.Fs + kFrontWaves - 1) / kFrontWaves), fb(kFrontThreads);
    if (T == 1) hipLaunchKernelGGL(few_front_kernel<1>, front, fb, 0, s, a);
    else if (T <= 4) hipLaunchKernelGGL(few_front_kernel<4>, front, fb, 0, s, a);
    else hipLaunchKernelGGL(few_front_kernel<16>, front, fb, 0, s, a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const dim3 grid(a.gateup_wgs + (a.H + kFewCols - 1) / kFewCols), block(kFewThreads);
    if (ex->gate.fmt == MOE_W_BF16) hipLaunchKernelGGL(few_experts_kernel<F_BF16>, grid, block, 0, s, a);
    else if (ex->gate.fmt == MOE_W_FP8_BLOCK) hipLaunchKernelGGL(few_experts_kernel<F_FP8>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(few_experts_kernel<F_AWQ>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
