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
//    itself from the logits (cheaper than a third launch or a wait).  All of
//    them then take gate/up items (an expert's columns) until none is left and
//    write gate_tj h; load their first down rows; wait until all items are done;
//    and sum the experts, and the shared expert, for their share of the outputs
//    in fp32, in a fixed order.  Up to five workgroups share the same 16 outputs;
//    the last of them to finish adds the parts, again in a fixed order.
//
// The wait always ends: it begins when no gate/up item is left untaken, so each
// of them is in the hands of a running workgroup, and those wait for nothing
// before they have finished it.  (No workgroup needs another to be resident
// that is not, whatever else runs on the GPU.)  It is bounded all the same, so
// that a second call which clears the workspace meanwhile cannot hang the GPU.
// Where the bound is met y is NaN, but that is no detection: such calls can as
// well read each other's h, or leave outputs unwritten; y is undefined.
// Items are counted in 16 ranges, a cache line each: one counter for all took
// 20 ns an item, more than the item's work.
// h passes between compute dies, whose L2s are not coherent within a kernel:
// stores of it go past them (agent scope, sc1) and have completed before their
// workgroup counts itself done; loads of it follow an acquire fence after the wait.
//
// The products run on the bf16 16 x 16 x 32 MFMA: 16 weight rows x the 16
// possible tokens, a token that is not routed to the expert reading zeros
// (without memory traffic).  Weights stream 16 bytes a lane: 8 bf16, 16 E4M3
// or 32 4-bit inputs of one row, widened to bf16 exactly; their scales are
// applied to the fp32 sums, so nothing is rounded but h and y, both to bf16.
// Against dot products on the vector units this is a fifth of the instructions,
// which counts twice at one token, where every instruction runs once and is
// fetched from memory.
//
// Measured, hidden 2560, 10 of 512 experts of 640, a shared expert of 640: one
// token in 38 (FP8), 39 (4-bit) and 48 us (bf16), of which the bytes need 13, 8
// and 24; the layer of separate kernels takes 55 to 63, 63 to 66 and 60 to 65.
// Four tokens take the same either way (71 to 101 us).  16 take 188 to 198, 182
// and 291 us here and 155 to 159, 117 to 121 and 250 to 255 there: of 188 the
// front took 12, selection 9, gate/up 98 (4.6 TB/s), the items' ends and the wait 11.
#include "fp8.h"
#include "ffn_internal.h"
#include "select.h"

namespace moe {

namespace {

constexpr int kFewThreads = 512, kFewWaves = kFewThreads / kWave;
constexpr int kFewMaxPairs = kFewMaxT * 64;
constexpr int kAgent = 16;         // cache policy of buffer accesses: sc1

enum { F_BF16 = 0, F_FP8 = 1, F_AWQ = 2 };

// Counters, 128 bytes apart: items taken of each range, items done of each
// range, ranges done; then, 4 bytes apart, finished workgroups of each 16 outputs.
constexpr int kRanges = 16;
constexpr int kFewSplits = 5;      // workgroups that can share 16 outputs
enum FewCount { C_TAKEN = 0, C_DONE = 32 * kRanges, C_ROOT = 64 * kRanges, C_OUT = 64 * kRanges + 32 };

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
    int down_wgs;           // workgroups that share the down pass
    uint32_t* counters;     // see FewCount
    float* parts;           // [kFewSplits][H / 16][16 x 16] sums of down workgroups
    float* logits;          // [T][E]
    uint16_t* hs;           // shared h [T][Fs] bf16
    uint16_t* h;            // gated h of every pair [T k][F] bf16
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

// The 16 rows of a fragment as one lane sees them: its row's bytes and its
// scales.  Gate/up fragments hold 8 columns of the gate's rows and the same 8 of
// the up's, so the addresses are per lane.
template <int FMT>
struct Rows {
    const uint8_t* w;     // the lane's row, at its piece of unit 0
    const float* s[2];    // E4M3: block scales of rows 0 .. 7 and 8 .. 15 (uniform)
    const uint16_t* gs;   // 4-bit: scales of rows 4 g .. + 3, one row of O per group of 32 inputs
    const uint8_t* gz;    // and their zero words
    int O;

    // row l % 16 of the fragment is output `o` of p (may differ by lane); rows
    // 4 g .. + 3 are outputs `o4` .. of p4; rows 0 .. 7 are of pa, the others of
    // pb, all outputs of one block of 128 with o0
    __device__ __forceinline__ void init(const FewProj& p, int o, const FewProj& p4, int o4, const FewProj& pa, const FewProj& pb,
                                         int o0, int e, int O_, int I, int lane) {
        using Un = Unit<FMT>;
        O = O_;
        const uint32_t rowb = (uint32_t)(I / 8) * Un::ROW8;
        w = static_cast<const uint8_t*>(p.w) + ((size_t)e * O + o) * rowb + 16 * (lane >> 4);
        if (FMT == F_FP8) {
            const size_t at = ((size_t)e * (O / 128) + o0 / 128) * (I / 128);
            s[0] = pa.bscales + at;
            s[1] = pb.bscales + at;
        }
        if (FMT == F_AWQ) {
            // lane l of 16 loads group l % 4 of a unit
            gs = p4.scales + ((size_t)e * (I / 32) + (lane & 3)) * O + o4;
            gz = reinterpret_cast<const uint8_t*>(p4.qzeros + ((size_t)e * (I / 32) + (lane & 3)) * (O / 8) + o4 / 8);
        }
    }
};

template <int FMT>
struct UnitData {
    i32x4_t w;
    float s[2];                   // E4M3 (uniform)
    u32x2_t gs;                   // 4-bit: four fp16 scales of a group
    uint32_t gz;                  // and their zero word
};

typedef const __attribute__((address_space(4))) float const_float;

// Unit u of the lane's row.
template <int FMT>
__device__ __forceinline__ void load_unit(UnitData<FMT>& d, const Rows<FMT>& r, int u) {
    d.w = *reinterpret_cast<const i32x4_t*>(r.w + 64 * (size_t)u);
    if (FMT == F_FP8) {
        d.s[0] = ((const_float*)r.s[0])[u / 2];
        d.s[1] = ((const_float*)r.s[1])[u / 2];
    }
    if (FMT == F_AWQ) {
        d.gs = *reinterpret_cast<const u32x2_t*>(r.gs + (size_t)(4 * u) * r.O);
        d.gz = *reinterpret_cast<const uint32_t*>(r.gz + (size_t)(4 * u) * (r.O / 2));
    }
}

// (v & mask) | c in one instruction: it takes one of the two constants from a
// scalar register, so c is kept in a vector register.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t c) {
    asm("" : "+v"(c));
    return (v & mask) | c;
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
            for (int i = 0; i < 4; ++i) v[i] = and_or(q[j] >> (4 * i), 0x000F000Fu, 0x43004300u);
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

// The value of lane J of each 16 (row_newbcast).
template <int J>
__device__ __forceinline__ uint32_t row_lane(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x150 + J, 0xF, 0xF, true);
}

// One group of a 4-bit unit: acc += s (sum (128 + q) x - (128 + z) sum x).
template <int J>
__device__ __forceinline__ void awq_group(f32x4_t& acc, const UnitData<F_AWQ>& d, bf16x8_t a, bf16x8_t b, int zshift) {
    const u32x4_t one4 = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    const f32x4_t zero = {};
    const f32x4_t v = mfma32(a, b, zero), sum = mfma32(__builtin_bit_cast(bf16x8_t, one4), b, zero);
    // zeros of rows 4 g + i: AWQ order of the word's nibbles
    const uint32_t zw = row_lane<J>(d.gz) >> zshift;  // 8 where rows 4 g .. are outputs 4 .. 7 of their word
    const uint32_t gs[2] = {row_lane<J>(d.gs[0]), row_lane<J>(d.gs[1])};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // 128 + z: its bits are 0x43000000 | z << 16
        const uint32_t zn = i == 0 ? zw << 16 : i == 1 ? zw : i == 2 ? zw << 12 : zw >> 4;
        const float z = __uint_as_float(and_or(zn, 0x000F0000u, 0x43000000u));
        const float s = f16_to_f32((gs[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
        acc[i] = fmaf(s, fmaf(-z, sum[i], v[i]), acc[i]);
    }
}

// acc += unit . inputs.
template <int FMT>
__device__ __forceinline__ void unit_product(f32x4_t& acc, const UnitData<FMT>& d, const bf16x8_t (&b)[Unit<FMT>::FRAGS],
                                             int zshift) {
    constexpr int FR = Unit<FMT>::FRAGS;
    bf16x8_t a[FR];
    unit_frags<FMT>(d, a);
    if constexpr (FMT == F_BF16) {
        acc = mfma32(a[0], b[0], acc);
    } else if constexpr (FMT == F_FP8) {
        f32x4_t v = {};
#pragma unroll
        for (int j = 0; j < FR; ++j) v = mfma32(a[j], b[j], v);
        const float s = threadIdx.x & 32 ? d.s[1] : d.s[0];  // rows 4 g ..: 8 and on from lane 32
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, v[i], acc[i]);
    } else {
        awq_group<0>(acc, d, a[0], b[0], zshift);
        awq_group<1>(acc, d, a[1], b[1], zshift);
        awq_group<2>(acc, d, a[2], b[2], zshift);
        awq_group<3>(acc, d, a[3], b[3], zshift);
    }
}

// LDS reads and writes of the workgroup's waves are ordered; loads from memory
// stay under way (unlike __syncthreads).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Units of a gate/up batch, under way at once.  The four waves of a SIMD hide
// one another's loads; longer batches cost registers and so waves (16 tokens,
// FP8: 226 us with two waves), and the next batch's weights loaded ahead gain
// nothing here (4-bit 195 against 188 us, FP8 188 both).
template <int FMT>
constexpr int kBatch = FMT == F_AWQ ? 2 : FMT == F_FP8 ? 5 : 10;

// Gate (rows 0..7) and up (rows 8..15) of 8 columns from o0 of expert e.
template <int FMT>
__device__ __forceinline__ Rows<FMT> gateup_rows(const FewProj& pg, const FewProj& pu, int e, int F, int H, int o0) {
    const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
    Rows<FMT> r;
    r.init(l16 < 8 ? pg : pu, o0 + (l16 & 7), g < 2 ? pg : pu, o0 + 4 * (g & 1), pg, pu, o0, e, F, H, lane);
    return r;
}

template <int FMT>
__device__ __forceinline__ void load_batch(UnitData<FMT> (&d)[kBatch<FMT>], const Rows<FMT>& r, int ub, int u1) {
#pragma unroll
    for (int i = 0; i < kBatch<FMT>; ++i)
        if (ub + i < u1) load_unit<FMT>(d[i], r, ub + i);
}

// acc += units u0 .. u1 - 1 times x of the tokens whose byte offset is xoff
// (kOob: none; token l).
template <int FMT>
__device__ __forceinline__ void gateup_units(f32x4_t& acc, const Rows<FMT>& r, __amdgpu_buffer_rsrc_t rx, uint32_t xoff, int u0,
                                             int u1) {
    using Un = Unit<FMT>;
    constexpr int FR = Un::FRAGS, U = kBatch<FMT>;
    const int g = (threadIdx.x & 63) >> 4;
    for (int ub = u0; ub < u1; ub += U) {
        UnitData<FMT> d[U];
        u32x4_t x[U][FR];
        load_batch<FMT>(d, r, ub, u1);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (ub + i < u1)
#pragma unroll
                for (int j = 0; j < FR; ++j)
                    x[i][j] = __builtin_bit_cast(
                        u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                     rx, xoff != kOob ? (int)(xoff + 2u * (uint32_t)((ub + i) * Un::IN + Un::input(g, j))) : (int)kOob,
                                     0, 0));
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (ub + i < u1) {
                bf16x8_t b[FR];
#pragma unroll
                for (int j = 0; j < FR; ++j) b[j] = input_frag<FMT>(x[i][j]);
                unit_product<FMT>(acc, d[i], b, 8 * (g & 1));
            }
    }
}

// The join of n waves' parts of such a fragment: lanes g < 2 get silu(gate) *
// up of columns o0 + 4 g .. of token l.
__device__ __forceinline__ f32x4_t gateup_join(const f32x4_t (*part)[kWave], int n, int lane) {
    f32x4_t v = part[0][lane], u = part[0][lane ^ 32], h;
    for (int q = 1; q < n; ++q) {
        v += part[q][lane];
        u += part[q][lane ^ 32];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = silu(v[i]) * u[i];
    return h;
}

// h of four neighbouring columns, rounded to bf16 as the layer of separate
// kernels does: kept in 16 bits more the down pass has twice the loads of it,
// and their number bounds that pass (16 tokens, FP8: 72 us against 58).
__device__ __forceinline__ void store_h(__amdgpu_buffer_rsrc_t r, uint32_t row, int F, int col, f32x4_t h, bool agent) {
    const u32x2_t a = {pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
    const uint32_t at = (row * (uint32_t)F + (uint32_t)col) * 2u;
    if (agent) __builtin_amdgcn_raw_buffer_store_b64(a, r, (int)at, 0, kAgent);
    else __builtin_amdgcn_raw_buffer_store_b64(a, r, (int)at, 0, 0);
}

// Units v0 .. v1 of the F inputs of a list of experts, one after another, into
// 16 outputs from o0.  expert(slot), hoff(slot): the slot's expert and the byte
// offset of the lane's token's h (kOob: not routed to it; the token's sum is
// then left alone, as zeros times the expert's weights are no zeros where those
// hold an infinity or a NaN).  `ready` is called once the first U units are under
// way.  The next U units' weights are loaded before the present ones are used
// (16 tokens, FP8: 205 -> 189 us, bf16 320 -> 285).
template <int FMT, int U, class Expert, class Hoff, class Ready>
__device__ __forceinline__ void down_units(f32x4_t& acc, const FewProj& pd, int H, int F, int o0, __amdgpu_buffer_rsrc_t rh,
                                           int v0, int v1, Expert expert, Hoff hoff, Ready ready) {
    using Un = Unit<FMT>;
    constexpr int FR = Un::FRAGS;
    const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
    const int n = F / Un::IN;
    auto load_w = [&](UnitData<FMT> (&d)[U], int vb) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (vb + i < v1) {
                const int v = vb + i, slot = v / n;
                Rows<FMT> r;
                r.init(pd, o0 + l16, pd, o0 + 4 * g, pd, pd, o0, expert(slot), H, F, lane);
                load_unit<FMT>(d[i], r, v - slot * n);
            }
    };
    UnitData<FMT> d[U], next[U];
    load_w(d, v0);
    ready();
    for (int vb = v0; vb < v1; vb += U) {
        u32x4_t h[U][FR];
        bool routed[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (vb + i < v1) {
                const int v = vb + i, slot = v / n;
                const uint32_t at = hoff(slot);
                routed[i] = at != kOob;
#pragma unroll
                for (int j = 0; j < FR; ++j) {
                    const uint32_t in = (uint32_t)((v - slot * n) * Un::IN + Un::input(g, j));
                    h[i][j] = __builtin_bit_cast(
                        u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rh, at != kOob ? (int)(at + 2u * in) : (int)kOob, 0, 0));
                }
            }
        load_w(next, vb + U);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (vb + i < v1) {
                bf16x8_t b[FR];
#pragma unroll
                for (int j = 0; j < FR; ++j) b[j] = input_frag<FMT>(h[i][j]);
                f32x4_t sum = acc;
                unit_product<FMT>(sum, d[i], b, 8 * (g & 1));
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[q] = routed[i] ? sum[q] : acc[q];
            }
#pragma unroll
        for (int i = 0; i < U; ++i) d[i] = next[i];
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
        for (int t = 0; t < kFrontTokens; ++t) if (t == 0 || t0 + t < a.T) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[t] = fma((double)__uint_as_float(r[i] << 16), (double)__uint_as_float(x[t][i] << 16), acc[t]);
                acc[t] = fma((double)__uint_as_float(r[i] & 0xFFFF0000u), (double)__uint_as_float(x[t][i] & 0xFFFF0000u), acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kFrontTokens; ++t) if (t0 + t < a.T) {
        const double s = wave_sum_f64(acc[t]);
        if (lane == 0) a.logits[(size_t)(t0 + t) * a.E + e] = (float)s;
    }
}

// The first Fs / 8 workgroups: 8 columns each of the shared expert's gate and
// up, the inputs split over the waves; the others: logits, one wave per expert
// and kFrontTokens tokens.
__global__ __launch_bounds__(kFewThreads, 4) void few_front_kernel(const FewArgs a) {
    __shared__ f32x4_t part[kFewWaves][kWave];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), l16 = lane & 15;
    if (blockIdx.x == 0) {
        for (int c = threadIdx.x; c < C_OUT + a.H / 16; c += kFewThreads) a.counters[c] = 0;
    }
    const int sh = a.Fs / 8;
    if ((int)blockIdx.x < sh) {
        const int o0 = blockIdx.x * 8;
        const __amdgpu_buffer_rsrc_t rx = fp8_rsrc(a.x, (uint32_t)a.T * (uint32_t)a.H * 2u);
        f32x4_t acc = {};
        const Rows<F_BF16> r = gateup_rows<F_BF16>(a.sgate, a.sup, 0, a.Fs, a.H, o0);
        const int n = a.H / Unit<F_BF16>::IN, u0 = n * wv / kFewWaves, u1 = n * (wv + 1) / kFewWaves;
        gateup_units<F_BF16>(acc, r, rx, l16 < a.T ? (uint32_t)(l16 * a.H) * 2u : kOob, u0, u1);
        part[wv][lane] = acc;
        __syncthreads();
        if (wv == 0 && lane < 32 && l16 < a.T) {
            f32x4_t h = gateup_join(part, kFewWaves, lane);
            const float s = a.shared_scale ? a.shared_scale[l16] : 1.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] *= s;
            store_h(fp8_rsrc(a.hs, (uint32_t)a.T * (uint32_t)a.Fs * 2u), (uint32_t)l16, a.Fs, o0 + 4 * (lane >> 4), h, false);
        }
        return;
    }
    const int w = (blockIdx.x - sh) * kFewWaves + wv, groups = (a.T + kFrontTokens - 1) / kFrontTokens;
    const int e = w / groups;
    if (e < a.E) front_logits(a, e, (w - e * groups) * kFrontTokens, lane);
}

// Lists of a workgroup in LDS, sized for the call (the fewer bytes, the more
// workgroups share a compute unit): P pairs, at most S touched experts.
struct FewLists {
    f32x4_t (*part)[kFewWaves][kWave];    // [2]
    uint2 (*cand)[kWave];                 // [waves], the selection's: in part, which is used after it
    uint32_t (*lane_max)[kWave];          // [waves], likewise
    int32_t* idx;                         // [P] expert of pair t k + j
    float* gate;                          // [P]
    int32_t* wave_slots;                  // [waves]
    int32_t* next;                        // [2]
    int32_t* mine;                        // [kRanges] items of each range this workgroup has done
    uint16_t (*pair)[kFewMaxT];           // [S] slot, token -> pair, or 0xFFFF
    uint16_t* slot_of;                    // [1024] expert -> slot
    uint16_t* expert;                     // [S] slot -> expert, ascending

    __host__ __device__ static constexpr size_t bytes(int P, int S) {
        return 2 * kFewWaves * kWave * 16 + (size_t)P * 8 + (kFewWaves + 2 + kRanges) * 4 +
               (size_t)S * kFewMaxT * 2 + 1024 * 2 + (size_t)S * 2;
    }
    __device__ __forceinline__ void place(uint8_t* m, int P, int S) {
        auto take = [&](size_t n) {
            uint8_t* at = m;
            m += n;
            return at;
        };
        part = reinterpret_cast<f32x4_t(*)[kFewWaves][kWave]>(take(2 * kFewWaves * kWave * 16));
        cand = reinterpret_cast<uint2(*)[kWave]>(part);
        lane_max = reinterpret_cast<uint32_t(*)[kWave]>(cand + kFewWaves);
        idx = reinterpret_cast<int32_t*>(take((size_t)P * 4));
        gate = reinterpret_cast<float*>(take((size_t)P * 4));
        wave_slots = reinterpret_cast<int32_t*>(take(kFewWaves * 4));
        next = reinterpret_cast<int32_t*>(take(2 * 4));
        mine = reinterpret_cast<int32_t*>(take(kRanges * 4));
        pair = reinterpret_cast<uint16_t(*)[kFewMaxT]>(take((size_t)S * kFewMaxT * 2));
        slot_of = reinterpret_cast<uint16_t*>(take(1024 * 2));
        expert = reinterpret_cast<uint16_t*>(take((size_t)S * 2));
    }
};
static_assert(FewLists::bytes(kFewMaxPairs, 1024) <= 64 * 1024, "what a launch gets without asking");

// Top k of token t's E <= 512 logits by one wave.  Lane i holds experts 8 i ..
// 8 i + 7.  Of the lanes' largest logits, those with fewer than k others above
// them are at least k; all of these are logits at or above the smallest of them,
// so that one bounds the top k from below.  It usually leaves little more than k
// candidates, and each finds its rank by comparing itself with the others.
// Against k rounds of a wave-wide maximum this has no long chain, and a third
// of the instructions, which every workgroup of the launch executes.
__device__ __forceinline__ void few_topk(const FewArgs& a, const FewLists& s, int t, u32x4_t l0, u32x4_t l1, int wv, int lane) {
    uint32_t key[8], m = 0;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        key[v] = 8 * lane + v < a.E ? expert_key(__uint_as_float(v < 4 ? l0[v & 3] : l1[v & 3])) : 0u;
        m = max(m, key[v]);
    }
    s.lane_max[wv][lane] = m;
    __builtin_amdgcn_wave_barrier();
    int above = 0;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        const uint4 o = reinterpret_cast<const uint4*>(s.lane_max[wv])[i];
        above += (o.x > m) + (o.y > m) + (o.z > m) + (o.w > m);
    }
    const uint32_t least = ~wave_max_u32(above < a.k ? ~m : 0u);
    int n = 0;
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        const bool is = key[v] >= least && key[v] != 0;
        const uint64_t b = __ballot(is);
        const int at = n + __popcll(b & below);
        if (is && at < kWave) s.cand[wv][at] = make_uint2(key[v], (uint32_t)(8 * lane + v));
        n += __popcll(b);
    }
    __builtin_amdgcn_wave_barrier();
    if (n > kWave) {  // many equal logits, or k near E: the rounds
        select_token<8>(a.logits, (size_t)t, a.E, a.k, a.k, lane, s.idx, nullptr, s.gate);
        return;
    }
    const uint2 mine = lane < n ? s.cand[wv][lane] : make_uint2(0u, 0xFFFFFFFFu);
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const uint2 o = s.cand[wv][i];
        rank += o.x > mine.x || (o.x == mine.x && o.y < mine.y);
    }
    const bool in = lane < n && rank < a.k;
    const float top = float_from_order_key(wave_max_u32(m));
    const float p = in ? expf(float_from_order_key(mine.x) - top) : 0.0f;
    const float z = wave_sum_f32(p);
    if (in) {
        s.idx[t * a.k + rank] = (int32_t)mine.y;
        s.gate[t * a.k + rank] = p / z;
    }
}

// Selection and grouping, the same in every workgroup: the top k of every
// token, then the touched experts in ascending order, and which pair of which
// token each of them has.  Returns the number of touched experts.
__device__ __forceinline__ int few_select(const FewArgs& a, const FewLists& s) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, P = a.T * a.k;
    for (int e = threadIdx.x; e < 1024; e += kFewThreads) s.slot_of[e] = 0;
    const int slots_max = min(P, a.E);
    for (int i = threadIdx.x; i < slots_max * (kFewMaxT / 2); i += kFewThreads)
        reinterpret_cast<uint32_t*>(s.pair)[i] = 0xFFFFFFFFu;
    static_assert(kFewMaxT == 2 * kFewWaves, "two tokens a wave");
    if (a.E <= 512) {
        u32x4_t l[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = min(wv + i * kFewWaves, a.T - 1);
            const __amdgpu_buffer_rsrc_t rl = fp8_rsrc(a.logits + (size_t)t * a.E, (uint32_t)a.E * 4u);
            l[i][0] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rl, lane * 32, 0, 0));
            l[i][1] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rl, lane * 32 + 16, 0, 0));
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            if (wv + i * kFewWaves < a.T) few_topk(a, s, wv + i * kFewWaves, l[0][0], l[0][1], wv, lane);
            l[0][0] = l[1][0];
            l[0][1] = l[1][1];
        }
    } else {
        for (int t = wv; t < a.T; t += kFewWaves)
            select_token<16>(a.logits, (size_t)t, a.E, a.k, a.k, lane, s.idx, nullptr, s.gate);
    }
    lds_barrier();
    for (int p = threadIdx.x; p < P; p += kFewThreads) s.slot_of[s.idx[p]] = 1;
    lds_barrier();
    // thread i numbers experts 2 i and 2 i + 1
    const uint32_t two = reinterpret_cast<const uint32_t*>(s.slot_of)[threadIdx.x];
    const uint64_t m0 = __ballot(two & 1u), m1 = __ballot(two >> 16);
    const uint64_t below = (1ull << lane) - 1;
    int at = __popcll(m0 & below) + __popcll(m1 & below);
    if (lane == 0) s.wave_slots[wv] = __popcll(m0) + __popcll(m1);
    lds_barrier();
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
    lds_barrier();
    for (int p = threadIdx.x; p < P; p += kFewThreads) s.pair[s.slot_of[s.idx[p]]][p / a.k] = (uint16_t)p;
    lds_barrier();
    return __builtin_amdgcn_readfirstlane(slots);
}

// Sizes of the ranges of n items: the first n % kRanges have one more.
__device__ __forceinline__ int range_size(int n, int r) { return n / kRanges + (r < n % kRanges); }
__device__ __forceinline__ int range_first(int n, int r) { return n / kRanges * r + min(r, n % kRanges); }

// Takes items for a workgroup (one wave): take() asks for the next of range `r`,
// take_result() is that item, or one of any range that has some left (r becomes
// that one), or -1 when all are taken.  They are apart because a wave's loads
// return in order: asked for before the weights are, the answer is there when
// they are.
__device__ __forceinline__ uint32_t take(const FewArgs& a, int r, int lane) {
    uint32_t v = 0;
    if (lane == 0)
        v = __hip_atomic_fetch_add(a.counters + C_TAKEN + 32 * r, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return v;
}

__device__ __forceinline__ int take_result(const FewArgs& a, int n, int& r, uint32_t v, int lane) {
    for (;;) {
        const uint32_t got = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
        if (got < (uint32_t)range_size(n, r)) return range_first(n, r) + (int)got;
        uint32_t c = 0xFFFFFFFFu;
        if (lane < kRanges)
            c = __hip_atomic_load(a.counters + C_TAKEN + 32 * lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint64_t left = __ballot(lane < kRanges && c < (uint32_t)range_size(n, lane));
        if (left == 0) return -1;
        // the next range after r, so that the searchers spread
        const uint64_t after = left & ~((2ull << r) - 1);
        r = __ffsll((long long)(after ? after : left)) - 1;
        v = take(a, r, lane);
    }
}

template <int FMT>
__global__ __launch_bounds__(kFewThreads, 4) void few_experts_kernel(const FewArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t few_smem[];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int l16 = lane & 15, g4 = 4 * (lane >> 4);
    const int P = a.T * a.k;
    FewLists s;
    s.place(few_smem, P, min(P, a.E));
    f32x4_t (*part)[kFewWaves][kWave] = s.part;
    if (threadIdx.x < kRanges) s.mine[threadIdx.x] = 0;
    int r = blockIdx.x % kRanges;
    uint32_t taken = 0;
    if (wv == 0) taken = take(a, r, lane);
    const int slots = few_select(a, s);
    const __amdgpu_buffer_rsrc_t rh = fp8_rsrc(a.h, (uint32_t)P * (uint32_t)a.F * 2u);

    // ---- gate/up.  An item is 8 columns of an expert for each group of `ks`
    // waves, which split the inputs and are joined in their order through LDS:
    // few items are cut finely, many keep a wave on longer runs, and the 4-bit
    // rows, half as long, take the coarser cut.  (Hidden 2560, 640 columns, cut in
    // 8 / 4 / 2.  16 tokens, about 138 experts: FP8 195 / 188 / 189 us, 4-bit 203 /
    // 187 / 179; 4 tokens: FP8 70 / 72 / -, 4-bit 74 / 71 / -; 1 token: FP8 37.9 /
    // 37.3 / 43.0, 4-bit 39.2 / 38.1 / 45.3, bf16 48.2 / 49.2 / 59.2.)
    const int cols8 = slots * (a.F / 8);
    const int ks = cols8 < 1024 ? 8 : cols8 < 4096 ? (FMT == F_AWQ ? 4 : 8) : FMT == F_AWQ ? 2 : 4;
    const int cw = kFewWaves / ks;
    const int per = (a.F / 8 + cw - 1) / cw, items = slots * per;
    const int ranges = min(items, kRanges);
    {
        using Un = Unit<FMT>;
        const __amdgpu_buffer_rsrc_t rx = fp8_rsrc(a.x, (uint32_t)a.T * (uint32_t)a.H * 2u);
        const int n = a.H / Un::IN, part_of = wv % ks, group = wv / ks;
        const int u0 = n * part_of / ks, u1 = n * (part_of + 1) / ks;
        if (wv == 0) {
            const int first = take_result(a, items, r, taken, lane);
            if (lane == 0) s.next[1] = first;
        }
        lds_barrier();
        int item = __builtin_amdgcn_readfirstlane(s.next[1]);
        // columns past F (F / 8 no multiple of the groups) repeat the last ones and are not stored
        auto first_col = [&](int it) { return (it % per * cw + group) * 8; };
        auto rows_of = [&](int it) {
            const int e = __builtin_amdgcn_readfirstlane((int)s.expert[it / per]);
            return gateup_rows<FMT>(a.gate, a.up, e, a.F, a.H, min(first_col(it), a.F - 8));
        };
        for (int buf = 0; item >= 0; buf ^= 1) {
            const uint32_t p = s.pair[item / per][l16];
            f32x4_t acc = {};
            if (wv == 0) taken = take(a, r, lane);  // the next one, before the weights' loads
            gateup_units<FMT>(acc, rows_of(item), rx, p != 0xFFFFu ? (uint32_t)(l16 * a.H) * 2u : kOob, u0, u1);
            part[buf][wv][lane] = acc;
            if (wv == 0) {
                const int next = take_result(a, items, r, taken, lane);
                if (lane == 0) {
                    s.next[buf] = next;
                    int q = 0;
                    while (q + 1 < ranges && item >= range_first(items, q + 1)) ++q;
                    ++s.mine[q];
                }
            }
            lds_barrier();
            const int next = __builtin_amdgcn_readfirstlane(s.next[buf]);
            if (part_of == 0 && lane < 32 && p != 0xFFFFu && first_col(item) < a.F) {
                f32x4_t h = gateup_join(&part[buf][wv], ks, lane);
                const float gate = s.gate[p];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] *= gate;
                store_h(rh, p, a.F, first_col(item) + g4, h, true);
            }
            item = next;
        }
        if (blockIdx.x == 0 && a.topk_idx)
            for (int p = threadIdx.x; p < P; p += kFewThreads) a.topk_idx[p] = s.idx[p];
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the stores have completed
        lds_barrier();
        if (wv == 0 && lane < ranges && s.mine[lane] > 0) {
            const uint32_t mine = (uint32_t)s.mine[lane];
            const uint32_t before =
                __hip_atomic_fetch_add(a.counters + C_DONE + 32 * lane, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (before + mine == (uint32_t)range_size(items, lane))
                __hip_atomic_fetch_add(a.counters + C_ROOT, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }

    // ---- down.  The units of all experts for 16 outputs, and those of all
    // groups of 16 outputs one after another, are one list, of which every
    // workgroup takes an equal run (at least a quarter of a group's units, so at
    // most kFewSplits share a group), and of its part of a group every wave.
    const int nc = a.H / 16, n = slots * (a.F / Unit<FMT>::IN);
    const int wgs = min(a.down_wgs, nc * min(n, kFewSplits - 1));  // no run is empty
    if ((int)blockIdx.x >= wgs) return;
    const int64_t all = (int64_t)nc * n;
    auto run_begin = [&](int b) { return all * b / wgs; };
    const int64_t v0 = run_begin(blockIdx.x), v1 = run_begin(blockIdx.x + 1);
    bool first = true, ok = true;
    auto ready = [&] {
        if (!first) return;
        first = false;
        // all ranges of items done?
        if (wv == 0) {
            const uint64_t begin = wall_clock64();
            for (;;) {
                const uint32_t v = __hip_atomic_load(a.counters + C_ROOT, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                if ((uint32_t)__builtin_amdgcn_readfirstlane((int)v) >= (uint32_t)ranges) break;
                if (wall_clock64() - begin > 400000000ull) {  // 4 s of the 100 MHz counter
                    ok = false;
                    break;
                }
                __builtin_amdgcn_s_sleep(4);
            }
            // what this compute unit and its die have cached of h is older
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        }
        lds_barrier();
    };
    int buf = 0;
    for (int64_t v = v0; v < v1; buf ^= 1) {
        const int c = (int)(v / n), o0 = c * 16;
        const int64_t cb = (int64_t)c * n, ce = v1 < cb + n ? v1 : cb + n;  // the run's units of this group: v .. ce
        const int b0 = (int)(v - cb), len = (int)(ce - v);
        f32x4_t acc = {};
        down_units<FMT, (FMT == F_FP8 ? 5 : FMT == F_AWQ ? 2 : 6)>(
            acc, a.down, a.H, a.F, o0, rh, b0 + len * wv / kFewWaves,
            b0 + len * (wv + 1) / kFewWaves, [&](int u) { return __builtin_amdgcn_readfirstlane((int)s.expert[u]); },
            [&](int u) {
                const uint32_t p = s.pair[u][l16];
                return p != 0xFFFFu ? p * (uint32_t)a.F * 2u : kOob;
            },
            ready);
        // the shared expert's part goes with the first unit of the group
        if (a.Fs && b0 == 0) {
            const int ns = a.Fs / Unit<F_BF16>::IN;
            down_units<F_BF16, 3>(
                acc, a.sdown, a.H, a.Fs, o0, fp8_rsrc(a.hs, (uint32_t)a.T * (uint32_t)a.Fs * 2u), ns * wv / kFewWaves, ns * (wv + 1) / kFewWaves, [](int) { return 0; },
                [&](int) { return l16 < a.T ? (uint32_t)(l16 * a.Fs) * 2u : kOob; }, [] {});
        }
        if (!ok) acc = f32x4_t{1, 1, 1, 1} * __uint_as_float(0x7FC00000u);
        part[buf][wv][lane] = acc;
        v = ce;
        lds_barrier();
        if (wv != 0) continue;
#pragma unroll
        for (int q = 1; q < kFewWaves; ++q) acc += part[buf][q][lane];
        // workgroups with units of this group: those whose runs hold its first to its last unit
        auto owner = [&](int64_t unit) {
            int b = (int)(unit * wgs / all);
            while (run_begin(b + 1) <= unit) ++b;
            while (run_begin(b) > unit) --b;
            return b;
        };
        const int wb = owner(cb), we = owner(cb + n - 1);
        if (wb != we) {
            // leave the sum, count; the last of the workgroups adds them all
            const __amdgpu_buffer_rsrc_t rp = fp8_rsrc(a.parts, (uint32_t)kFewSplits * (uint32_t)nc * 1024u);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc), rp,
                                                   (((int)blockIdx.x - wb) * nc + c) * 1024 + lane * 16, 0, kAgent);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            uint32_t before = 0;
            if (lane == 0)
                before = __hip_atomic_fetch_add(a.counters + C_OUT + c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (__builtin_amdgcn_readfirstlane((int)before) != we - wb) continue;
            asm volatile("" ::: "memory");
            acc = f32x4_t{};
            for (int q = 0; q <= we - wb; ++q)
                acc += __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rp, (q * nc + c) * 1024 + lane * 16, 0,
                                                                                        kAgent));
        }
        if (l16 < a.T)
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

static size_t few_counter_bytes(int H) { return up256((C_OUT + (size_t)H / 16) * 4); }

size_t few_ws_bytes(int T, int k, const moe_experts* ex, const moe_experts* sh) {
    return few_counter_bytes(ex->hidden) + up256((size_t)kFewSplits * (ex->hidden / 16) * 1024) +
           up256((size_t)T * ex->num_experts * 4) + up256(sh ? (size_t)T * sh->inter * 2 : 0) +
           up256((size_t)T * k * ex->inter * 2);
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
    w += few_counter_bytes(a.H);
    a.parts = reinterpret_cast<float*>(w);
    w += up256((size_t)kFewSplits * (a.H / 16) * 1024);
    a.logits = reinterpret_cast<float*>(w);
    w += up256((size_t)T * a.E * 4);
    a.hs = reinterpret_cast<uint16_t*>(w);
    w += up256((size_t)T * a.Fs * 2);
    a.h = reinterpret_cast<uint16_t*>(w);
    a.y = y;
    a.topk_idx = topk_idx;
    // two workgroups a compute unit, which the registers allow; fewer where there is less to do
    const int nc = a.H / 16;
    a.down_wgs = nc * (kFewSplits - 1) < 512 ? nc * (kFewSplits - 1) : 512;
    const int most = T * k < a.E ? T * k : a.E;
    const long items = (long)most * (a.F / 8);
    const int wgs = items < 512 ? (int)items : 512;
    const size_t lds = FewLists::bytes(T * k, most);
    const int groups = (T + kFrontTokens - 1) / kFrontTokens;
    const dim3 front(a.Fs / 8 + (a.E * groups + kFewWaves - 1) / kFewWaves), block(kFewThreads);
    hipLaunchKernelGGL(few_front_kernel, front, block, 0, s, a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const dim3 grid(wgs > a.down_wgs ? wgs : a.down_wgs);
    if (ex->gate.fmt == MOE_W_BF16) hipLaunchKernelGGL(few_experts_kernel<F_BF16>, grid, block, lds, s, a);
    else if (ex->gate.fmt == MOE_W_FP8_BLOCK) hipLaunchKernelGGL(few_experts_kernel<F_FP8>, grid, block, lds, s, a);
    else hipLaunchKernelGGL(few_experts_kernel<F_AWQ>, grid, block, lds, s, a);
    return hipGetLastError();
}

}  // namespace moe
