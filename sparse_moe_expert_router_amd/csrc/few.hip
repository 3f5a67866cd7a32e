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
//    a ticket.  The first tickets are gate/up workgroups: they write gate_tj h
//    and count themselves done.  The others own 16 outputs each: they do their
//    part of the shared expert, load their first down rows, wait for the
//    count, and sum all experts in fp32, in a fixed order.
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
// The products run on the bf16 16 x 16 x 32 MFMA: 16 weight rows x the 16
// possible tokens, a token that is not routed to the expert reading zeros
// (without memory traffic).  Weights stream 16 bytes a lane: 8 bf16, 16 E4M3
// or 32 4-bit inputs of one row, widened to bf16 exactly; their scales are
// applied to the fp32 sums, so nothing is rounded but h, kept as the sum of
// two bf16 (16 bits of mantissa), and y.  Against dot products on the vector
// units this is a fifth of the instructions, which counts twice at one token,
// where every instruction runs once and is fetched from memory.
#include "fp8.h"
#include "ffn_internal.h"
#include "select.h"

namespace moe {

namespace {

constexpr int kFewThreads = 512, kFewWaves = kFewThreads / kWave;
constexpr int kFewMaxPairs = kFewMaxT * 64;
constexpr int kAgent = 16;         // cache policy of buffer accesses: sc1
constexpr int kStream = 2;         // non-temporal

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
    uint16_t* hs;           // shared h: bf16 parts [2][T][Fs]
    uint16_t* h;            // gated h of every pair: bf16 parts [2][T k][F]
    uint16_t* y;            // [T][H]
    int32_t* topk_idx;      // [T][k] or nullptr
};

// A unit is what 64 lanes load of 16 rows with 16 bytes each: lane 16 g + l
// holds row l.  It feeds FRAGS MFMAs; input 8 bytes.. of lane group g in MFMA j:
//   bf16  (32 inputs):  8 g
//   E4M3  (64 inputs):  16 g + 8 j
//   4-bit (128 inputs): 32 j + 8 g   (after an exchange between lane groups)
template <int FMT>
struct Unit {
    static constexpr int IN = FMT == F_BF16 ? 32 : FMT == F_FP8 ? 64 : 128;
    static constexpr int FRAGS = FMT == F_BF16 ? 1 : FMT == F_FP8 ? 2 : 4;
    static constexpr int ROW8 = FMT == F_BF16 ? 16 : FMT == F_FP8 ? 8 : 4;  // bytes of 8 inputs
    __device__ static __forceinline__ int input(int g, int j) {
        return FMT == F_BF16 ? 8 * g : FMT == F_FP8 ? 16 * g + 8 * j : 32 * j + 8 * g;
    }
};

// 16 rows (outputs o0 ..) of one expert's projection.
template <int FMT>
struct Rows {
    __amdgpu_buffer_rsrc_t w, s, z;
    uint32_t woff, soff, zoff;
    int O;

    __device__ __forceinline__ void init(const FewProj& p, int e, int O_, int I, int o0, int lane) {
        using Un = Unit<FMT>;
        O = O_;
        const uint32_t rowb = (uint32_t)(I / 8) * Un::ROW8;
        const size_t row = (size_t)e * O + o0;
        w = fp8_rsrc(static_cast<const uint8_t*>(p.w) + row * rowb, 16u * rowb);
        woff = (uint32_t)(lane & 15) * rowb + 16u * (uint32_t)(lane >> 4);
        if (FMT == F_FP8) {
            const int KB = I / 128;
            s = fp8_rsrc(p.bscales + ((size_t)e * (O / 128) + o0 / 128) * KB, (uint32_t)KB * 4u);
            soff = 0;
        }
        if (FMT == F_AWQ) {
            // scales and zeros of outputs o0 + 4 g .. + 3, one row of them per group of 32 inputs
            s = fp8_rsrc(p.scales + (size_t)e * (I / 32) * O, (uint32_t)(I / 32) * (uint32_t)O * 2u);
            z = fp8_rsrc(p.qzeros + (size_t)e * (I / 32) * (O / 8), (uint32_t)(I / 32) * (uint32_t)O / 2u);
            soff = (uint32_t)(o0 + 4 * (lane >> 4)) * 2u;
            zoff = (uint32_t)((o0 + 4 * (lane >> 4)) >> 3) * 4u;
        }
    }
};

template <int FMT>
struct UnitData {
    i32x4_t w;
    float s;                      // E4M3
    u32x2_t gs[4];                // 4-bit: four fp16 scales per group
    uint32_t gz[4];               // and their zero words
};

// Unit u; past the end (u >= n) everything reads zero.
template <int FMT>
__device__ __forceinline__ void load_unit(UnitData<FMT>& d, const Rows<FMT>& r, int u, int n) {
    const bool in = u < n;
    d.w = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r.w, in ? (int)(r.woff + 64u * u) : (int)kOob, 0, kStream));
    if (FMT == F_FP8) d.s = buf_load_f32(r.s, in ? (uint32_t)(u / 2) * 4u : kOob, 0);
    if (FMT == F_AWQ) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t so = r.soff + (uint32_t)(4 * u + j) * (uint32_t)r.O * 2u;
            const uint32_t zo = r.zoff + (uint32_t)(4 * u + j) * (uint32_t)r.O / 2u;
            d.gs[j] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r.s, in ? (int)so : (int)kOob, 0, 0));
            d.gz[j] = __builtin_amdgcn_raw_buffer_load_b32(r.z, in ? (int)zo : (int)kOob, 0, 0);
        }
    }
}

// The MFMA operands of a unit's weights.
template <int FMT>
__device__ __forceinline__ void unit_frags(const UnitData<FMT>& d, bf16x8_t (&a)[Unit<FMT>::FRAGS]) {
    if constexpr (FMT == F_BF16) {
        a[0] = __builtin_bit_cast(bf16x8_t, d.w);
    } else if constexpr (FMT == F_FP8) {
        a[0] = fp8_to_bf16x8(d.w[0], d.w[1]);
        a[1] = fp8_to_bf16x8(d.w[2], d.w[3]);
    } else {
        // lane group g holds the four words of group g; MFMA j wants word g of
        // group j in lane group g: a 4 x 4 transposition between lane groups
        uint32_t q[4] = {(uint32_t)d.w[0], (uint32_t)d.w[1], (uint32_t)d.w[2], (uint32_t)d.w[3]};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto t = __builtin_amdgcn_permlane32_swap(q[i], q[i + 2], false, false);
            q[i] = t[0];
            q[i + 2] = t[1];
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const auto t = __builtin_amdgcn_permlane16_swap(q[i], q[i + 1], false, false);
            q[i] = t[0];
            q[i + 1] = t[1];
        }
        // 128 + q is exact in bf16 (bits 0x4300 | q); inputs in the order 0,4,1,5,2,6,3,7
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u32x4_t v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = ((q[j] >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
            a[j] = __builtin_bit_cast(bf16x8_t, v);
        }
    }
}

// Eight bf16 inputs as an MFMA operand beside unit_frags' order.
template <int FMT>
__device__ __forceinline__ bf16x8_t input_frag(u32x4_t x) {
    if (FMT == F_AWQ) {
        const u32x4_t v = {__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                           __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
        return __builtin_bit_cast(bf16x8_t, v);
    }
    return __builtin_bit_cast(bf16x8_t, x);
}

__device__ __forceinline__ f32x4_t mfma32(bf16x8_t a, bf16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// acc += unit . inputs; b[NB][FRAGS]: the inputs are the sum of NB parts.
template <int FMT, int NB>
__device__ __forceinline__ void unit_product(f32x4_t& acc, const UnitData<FMT>& d, const bf16x8_t (&b)[NB][Unit<FMT>::FRAGS]) {
    constexpr int FR = Unit<FMT>::FRAGS;
    bf16x8_t a[FR];
    unit_frags<FMT>(d, a);
    if constexpr (FMT == F_BF16) {
#pragma unroll
        for (int p = 0; p < NB; ++p) acc = mfma32(a[0], b[p][0], acc);
    } else if constexpr (FMT == F_FP8) {
        f32x4_t v = {};
#pragma unroll
        for (int j = 0; j < FR; ++j)
#pragma unroll
            for (int p = 0; p < NB; ++p) v = mfma32(a[j], b[p][j], v);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(d.s, v[i], acc[i]);
    } else {
        // per group of 32: s (sum (128 + q) x - (128 + z) sum x), the second sum by ones
        const u32x4_t one4 = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, one4);
#pragma unroll
        for (int j = 0; j < FR; ++j) {
            f32x4_t v = {}, sum = {};
#pragma unroll
            for (int p = 0; p < NB; ++p) {
                v = mfma32(a[j], b[p][j], v);
                sum = mfma32(ones, b[p][j], sum);
            }
            // zeros of outputs 4 g + i: AWQ order of the word's nibbles
            const uint32_t zw = d.gz[j] >> ((threadIdx.x & 16) ? 8 : 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float z = (float)((zw >> ((i & 1) * 16 + (i >> 1) * 4)) & 15u) + 128.0f;
                const float s = f16_to_f32((d.gs[j][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
                acc[i] = fmaf(s, fmaf(-z, sum[i], v[i]), acc[i]);
            }
        }
    }
}

// LDS reads and writes of the workgroup's waves are ordered; loads from memory
// stay under way (unlike __syncthreads).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Gate and up of 16 columns for the tokens whose byte offset of x is `xoff`
// (kOob: none; one token a lane l), over the wave's share of the units.
template <int FMT>
__device__ __forceinline__ void gateup_units(f32x4_t (&acc)[2], const FewProj& pg, const FewProj& pu, int e, int F, int H,
                                             int o0, __amdgpu_buffer_rsrc_t rx, uint32_t xoff, int part, int parts) {
    using Un = Unit<FMT>;
    constexpr int U = FMT == F_AWQ ? 2 : 5, FR = Un::FRAGS;  // units under way
    const int lane = threadIdx.x & 63, g = lane >> 4;
    Rows<FMT> rg, ru;
    rg.init(pg, e, F, H, o0, lane);
    ru.init(pu, e, F, H, o0, lane);
    const int n = (H + Un::IN - 1) / Un::IN;
    const int u0 = n * part / parts, u1 = n * (part + 1) / parts;
    for (int ub = u0; ub < u1; ub += U) {
        UnitData<FMT> dg[U], du[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            load_unit<FMT>(dg[i], rg, ub + i, u1);
            load_unit<FMT>(du[i], ru, ub + i, u1);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            bf16x8_t b[1][FR];
#pragma unroll
            for (int j = 0; j < FR; ++j) {
                const uint32_t in = (uint32_t)((ub + i) * Un::IN + Un::input(g, j));
                const bool ok = ub + i < u1 && xoff != kOob;
                b[0][j] = input_frag<FMT>(__builtin_bit_cast(
                    u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rx, ok ? (int)(xoff + 2u * in) : (int)kOob, 0, 0)));
            }
            unit_product<FMT, 1>(acc[0], dg[i], b);
            unit_product<FMT, 1>(acc[1], du[i], b);
        }
    }
}

// h of four neighbouring columns as two bf16 parts, [2][rows][F].
__device__ __forceinline__ void store_h(__amdgpu_buffer_rsrc_t r, uint32_t row, uint32_t rows, int F, int col, f32x4_t h,
                                        int policy) {
    float lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = h[i] - bf16_to_f32(f32_to_bf16_bits(h[i]));
    const u32x2_t a = {pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
    const u32x2_t b = {pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3])};
    const uint32_t at = (row * (uint32_t)F + (uint32_t)col) * 2u;
    if (policy) {
        __builtin_amdgcn_raw_buffer_store_b64(a, r, (int)at, 0, kAgent);
        __builtin_amdgcn_raw_buffer_store_b64(b, r, (int)(at + rows * (uint32_t)F * 2u), 0, kAgent);
    } else {
        __builtin_amdgcn_raw_buffer_store_b64(a, r, (int)at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b64(b, r, (int)(at + rows * (uint32_t)F * 2u), 0, 0);
    }
}

// A part of 16 outputs of one expert: units part, ... of its F inputs for the
// tokens whose byte offset of h is `hoff` (kOob: none); lo: bytes to the second
// bf16 part.  D units are loaded before `ready` is called.
template <int FMT, int U, class Ready>
__device__ __forceinline__ void down_units(f32x4_t& acc, const FewProj& pd, int e, int H, int F, int o0,
                                           __amdgpu_buffer_rsrc_t rh, uint32_t hoff, uint32_t lo, int part, int parts,
                                           Ready ready) {
    using Un = Unit<FMT>;
    constexpr int FR = Un::FRAGS;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    Rows<FMT> rd;
    rd.init(pd, e, H, F, o0, lane);
    const int n = (F + Un::IN - 1) / Un::IN;
    const int u0 = n * part / parts, u1 = n * (part + 1) / parts;
    for (int ub = u0; ub < u1; ub += U) {
        UnitData<FMT> d[U];
#pragma unroll
        for (int i = 0; i < U; ++i) load_unit<FMT>(d[i], rd, ub + i, u1);
        ready();
#pragma unroll
        for (int i = 0; i < U; ++i) {
            bf16x8_t b[2][FR];
#pragma unroll
            for (int j = 0; j < FR; ++j) {
                const uint32_t in = (uint32_t)((ub + i) * Un::IN + Un::input(g, j));
                const bool ok = ub + i < u1 && hoff != kOob;
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    b[p][j] = input_frag<FMT>(__builtin_bit_cast(
                        u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rh, ok ? (int)(hoff + 2u * in + p * lo) : (int)kOob, 0,
                                                                       kAgent)));
            }
            unit_product<FMT, 2>(acc, d[i], b);
        }
    }
}

constexpr int kFrontTokens = 4;  // tokens of a wave

// Logits of one expert for kFrontTokens tokens from t0: exact bf16 products summed in fp64.
__device__ __forceinline__ void front_logits(const FewArgs& a, int e, int t0, int lane) {
    double acc[kFrontTokens];
#pragma unroll
    for (int t = 0; t < kFrontTokens; ++t) acc[t] = 0.0;
#pragma unroll 5
    for (int c = lane * 8; c < a.H; c += kWave * 8) {
        const u32x4_t r = *reinterpret_cast<const u32x4_t*>(a.router + (size_t)e * a.H + c);
        u32x4_t x[kFrontTokens];
#pragma unroll
        for (int t = 0; t < kFrontTokens; ++t)
            if (t == 0 || t0 + t < a.T) x[t] = *reinterpret_cast<const u32x4_t*>(a.x + (size_t)(t0 + t) * a.H + c);
#pragma unroll
        for (int t = 0; t < kFrontTokens; ++t) {
            if (t > 0 && t0 + t >= a.T) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[t] = fma((double)__uint_as_float(r[i] << 16), (double)__uint_as_float(x[t][i] << 16), acc[t]);
                acc[t] = fma((double)__uint_as_float(r[i] & 0xFFFF0000u), (double)__uint_as_float(x[t][i] & 0xFFFF0000u), acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kFrontTokens; ++t) {
        if (t0 + t >= a.T) break;
        const double s = wave_sum_f64(acc[t]);
        if (lane == 0) a.logits[(size_t)(t0 + t) * a.E + e] = (float)s;
    }
}

// The first Fs / 16 workgroups: 16 columns each of the shared expert's gate and
// up, the inputs split over the waves; the others: logits, one wave per expert
// and kFrontTokens tokens.
__global__ __launch_bounds__(kFewThreads, 4) void few_front_kernel(const FewArgs a) {
    __shared__ f32x4_t part[kFewWaves][2][kWave];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), l16 = lane & 15;
    if (blockIdx.x == 0 && threadIdx.x < 9) a.counters[32 * threadIdx.x] = 0;
    const int sh = a.Fs / 16;
    if ((int)blockIdx.x < sh) {
        const int o0 = blockIdx.x * 16;
        const __amdgpu_buffer_rsrc_t rx = fp8_rsrc(a.x, (uint32_t)a.T * (uint32_t)a.H * 2u);
        f32x4_t acc[2] = {};
        gateup_units<F_BF16>(acc, a.sgate, a.sup, 0, a.Fs, a.H, o0, rx, l16 < a.T ? (uint32_t)(l16 * a.H) * 2u : kOob, wv,
                             kFewWaves);
        part[wv][0][lane] = acc[0];
        part[wv][1][lane] = acc[1];
        __syncthreads();
        if (wv == 0 && l16 < a.T) {
            f32x4_t g = acc[0], u = acc[1], h;
#pragma unroll
            for (int q = 1; q < kFewWaves; ++q) {
                g += part[q][0][lane];
                u += part[q][1][lane];
            }
            const float s = a.shared_scale ? a.shared_scale[l16] : 1.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = silu(g[i]) * u[i] * s;
            store_h(fp8_rsrc(a.hs, (uint32_t)a.T * (uint32_t)a.Fs * 4u), (uint32_t)l16, (uint32_t)a.T, a.Fs,
                    o0 + 4 * (lane >> 4), h, 0);
        }
        return;
    }
    const int w = (blockIdx.x - sh) * kFewWaves + wv, groups = (a.T + kFrontTokens - 1) / kFrontTokens;
    const int e = w / groups;
    if (e < a.E) front_logits(a, e, (w - e * groups) * kFrontTokens, lane);
}

struct FewLists {
    int32_t idx[kFewMaxPairs];              // expert of pair t k + j
    float gate[kFewMaxPairs];
    uint16_t slot_of[1024];                 // expert -> slot
    uint16_t expert[kFewMaxPairs];          // slot -> expert, ascending
    uint16_t pair[kFewMaxPairs][kFewMaxT];  // slot, token -> pair, or 0xFFFF
    int32_t wave_slots[kFewWaves];
    int32_t ticket;
};

// Selection and grouping, the same in every workgroup: the top k of every
// token, then the touched experts in ascending order, and which pair of which
// token each of them has.  Returns the number of touched experts.
__device__ __forceinline__ int few_select(const FewArgs& a, FewLists& s) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, P = a.T * a.k;
    for (int e = threadIdx.x; e < 1024; e += kFewThreads) s.slot_of[e] = 0;
    const int slots_max = min(P, a.E);
    for (int i = threadIdx.x; i < slots_max * (kFewMaxT / 2); i += kFewThreads)
        reinterpret_cast<uint32_t*>(s.pair)[i] = 0xFFFFFFFFu;
    for (int t = wv; t < a.T; t += kFewWaves) {
        if (a.E <= 512) select_token<8>(a.logits, (size_t)t, a.E, a.k, a.k, lane, s.idx, nullptr, s.gate);
        else select_token<16>(a.logits, (size_t)t, a.E, a.k, a.k, lane, s.idx, nullptr, s.gate);
    }
    __syncthreads();
    for (int p = threadIdx.x; p < P; p += kFewThreads) s.slot_of[s.idx[p]] = 1;
    __syncthreads();
    // thread i numbers experts 2 i and 2 i + 1
    const uint32_t two = reinterpret_cast<const uint32_t*>(s.slot_of)[threadIdx.x];
    const uint64_t m0 = __ballot(two & 1u), m1 = __ballot(two >> 16);
    const uint64_t below = (1ull << lane) - 1;
    int at = __popcll(m0 & below) + __popcll(m1 & below);
    if (lane == 0) s.wave_slots[wv] = __popcll(m0) + __popcll(m1);
    __syncthreads();
    int slots = 0;
#pragma unroll
    for (int q = 0; q < kFewWaves; ++q) {
        if (q < wv) at += s.wave_slots[q];
        slots += s.wave_slots[q];
    }
    if (two & 1u) {
        s.slot_of[2 * threadIdx.x] = (uint16_t)at;
        s.expert[at++] = (uint16_t)(2 * threadIdx.x);
    }
    if (two >> 16) {
        s.slot_of[2 * threadIdx.x + 1] = (uint16_t)at;
        s.expert[at] = (uint16_t)(2 * threadIdx.x + 1);
    }
    __syncthreads();
    for (int p = threadIdx.x; p < P; p += kFewThreads) s.pair[s.slot_of[s.idx[p]]][p / a.k] = (uint16_t)p;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(slots);
}

template <int FMT>
__global__ __launch_bounds__(kFewThreads, 4) void few_experts_kernel(const FewArgs a) {
    __shared__ FewLists s;
    __shared__ f32x4_t part[2][kFewWaves][2][kWave];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int l16 = lane & 15, g4 = 4 * (lane >> 4);
    const int P = a.T * a.k;
    if (threadIdx.x == 0)
        s.ticket = (int)__hip_atomic_fetch_add(a.counters, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int slots = few_select(a, s);
    const int ticket = __builtin_amdgcn_readfirstlane(s.ticket);
    const __amdgpu_buffer_rsrc_t rh = fp8_rsrc(a.h, (uint32_t)P * (uint32_t)a.F * 4u);

    if (ticket < a.gateup_wgs) {
        // items (expert, 16 columns), the inputs split over the 8 waves and
        // joined in their order through LDS
        const __amdgpu_buffer_rsrc_t rx = fp8_rsrc(a.x, (uint32_t)a.T * (uint32_t)a.H * 2u);
        const int per = a.F / 16, n = slots * per;
        int buf = 0;
        for (int q = ticket; q < n; q += a.gateup_wgs, buf ^= 1) {
            const int u = q / per, o0 = (q - u * per) * 16;
            const uint32_t p = s.pair[u][l16];
            const int e = __builtin_amdgcn_readfirstlane((int)s.expert[u]);
            f32x4_t acc[2] = {};
            gateup_units<FMT>(acc, a.gate, a.up, e, a.F, a.H, o0, rx, p != 0xFFFFu ? (uint32_t)(l16 * a.H) * 2u : kOob, wv,
                              kFewWaves);
            part[buf][wv][0][lane] = acc[0];
            part[buf][wv][1][lane] = acc[1];
            lds_barrier();
            if (wv == 0 && p != 0xFFFFu) {
                f32x4_t g = acc[0], v = acc[1], h;
#pragma unroll
                for (int i = 1; i < kFewWaves; ++i) {
                    g += part[buf][i][0][lane];
                    v += part[buf][i][1][lane];
                }
                const float gate = s.gate[p];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = silu(g[i]) * v[i] * gate;
                store_h(rh, p, (uint32_t)P, a.F, o0 + g4, h, 1);
            }
        }
        if (ticket == 0 && a.topk_idx)
            for (int p = threadIdx.x; p < P; p += kFewThreads) a.topk_idx[p] = s.idx[p];
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the stores have completed
        __syncthreads();
        if (threadIdx.x == 0)
            __hip_atomic_fetch_add(a.counters + 32 * (1 + ticket % 8), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return;
    }

    // ---- outputs o0 .. o0 + 15, experts dealt over the waves
    const int o0 = (ticket - a.gateup_wgs) * 16;
    f32x4_t acc = {};
    if (a.Fs)
        down_units<F_BF16, 3>(acc, a.sdown, 0, a.H, a.Fs, o0, fp8_rsrc(a.hs, (uint32_t)a.T * (uint32_t)a.Fs * 4u),
                              l16 < a.T ? (uint32_t)(l16 * a.Fs) * 2u : kOob, (uint32_t)a.T * (uint32_t)a.Fs * 2u, wv,
                              kFewWaves, [] {});
    bool waited = false, ok = true;
    auto ready = [&] {
        // all gate/up workgroups done?  Lanes 0..7 read the eight counts.
        if (waited) return;
        waited = true;
        const uint64_t begin = wall_clock64();
        for (;;) {
            uint32_t c = 0;
            if (lane < 8) c = __hip_atomic_load(a.counters + 32 * (1 + lane), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int m = 4; m >= 1; m >>= 1) c += __shfl_xor(c, m, kWave);
            if ((uint32_t)__builtin_amdgcn_readfirstlane((int)c) >= (uint32_t)a.gateup_wgs) break;
            if (wall_clock64() - begin > 400000000ull) {  // 4 s of the 100 MHz counter
                ok = false;
                break;
            }
            __builtin_amdgcn_s_sleep(8);
        }
        asm volatile("" ::: "memory");
    };
    constexpr int U = FMT == F_AWQ ? 2 : 10;
    for (int u = wv; u < slots; u += kFewWaves) {
        const uint32_t p = s.pair[u][l16];
        const int e = __builtin_amdgcn_readfirstlane((int)s.expert[u]);
        down_units<FMT, U>(acc, a.down, e, a.H, a.F, o0, rh, p != 0xFFFFu ? p * (uint32_t)a.F * 2u : kOob,
                           (uint32_t)P * (uint32_t)a.F * 2u, 0, 1, ready);
    }
    if (!ok) acc = f32x4_t{1, 1, 1, 1} * __uint_as_float(0x7FC00000u);
    part[0][wv][0][lane] = acc;
    __syncthreads();
    if (wv == 0 && l16 < a.T) {
#pragma unroll
        for (int q = 1; q < kFewWaves; ++q) acc += part[0][q][0][lane];
        *reinterpret_cast<uint2*>(a.y + (size_t)l16 * a.H + o0 + g4) =
            make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
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
    a.hs = reinterpret_cast<uint16_t*>(w);
    w += up256((size_t)T * a.Fs * 4);
    a.h = reinterpret_cast<uint16_t*>(w);
    a.y = y;
    a.topk_idx = topk_idx;
    // at most two gate/up workgroups a compute unit, and no more than there can be items
    const long items = (long)(T * k < a.E ? T * k : a.E) * (a.F / 16);
    a.gateup_wgs = (int)(items < 512 ? items : 512);
    const int groups = (T + kFrontTokens - 1) / kFrontTokens;
    const dim3 front(a.Fs / 16 + (a.E * groups + kFewWaves - 1) / kFewWaves), block(kFewThreads);
    hipLaunchKernelGGL(few_front_kernel, front, block, 0, s, a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const dim3 grid(a.gateup_wgs + a.H / 16);
    if (ex->gate.fmt == MOE_W_BF16) hipLaunchKernelGGL(few_experts_kernel<F_BF16>, grid, block, 0, s, a);
    else if (ex->gate.fmt == MOE_W_FP8_BLOCK) hipLaunchKernelGGL(few_experts_kernel<F_FP8>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(few_experts_kernel<F_AWQ>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
