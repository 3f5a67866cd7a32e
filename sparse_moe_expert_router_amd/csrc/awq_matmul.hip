// Product of few bf16 rows with one AWQ matrix (4-bit codes, zeros and fp16
// scales per group of 32, 64 or 128 inputs, in GEMM packing):
//   y[m][n] = sum_g s[g][n] * sum_{i in g} x[m][i] (q[i][n] - z[g][n])
//
// Bound by the codes' bytes for large matrices (16 rows x 16384 x 16384: 36 us,
// 4.4 TB/s with the scales; one row 32 us), by the launch and one or two round
// trips to memory for small ones (one row x 2560 x 2560: 6.2 us).
//
// A word holds one input of 8 columns, so a lane that reads the words of 8
// consecutive inputs holds, for each of the word's 8 columns, 8 inputs: its
// operand of a 16 x 16 x 32 bf16 MFMA for that column (16 lanes: 16 words, 128
// columns; 4 groups of 16 lanes: 4 x 8 inputs).  Two
// v_perm bring the halves of two inputs' words together, then a shift and a
// v_and_or make the exact bf16 pair 16 + q of one column.  With fp32 sums
//   sum x (q - z) = sum x (16 + q) - (16 + z) sum x,
// sum x from one more MFMA whose second operand is ones, so that it lies in the
// lanes as the products do.  (128 + q would save one shift in four, at eight
// times the cancellation.)  The scale is applied in fp32.
//
// Up to four rows (awq_few_kernel): the four groups of lanes take four
// different runs of 32 inputs ("sets"), and the MFMA's 16 rows are 4 sets x 4
// rows of x, with zeros where a row's set is not the lanes' own.  Four steps of
// 8 inputs a set then sum up in the MFMA's accumulator, and each lane scales only the
// sums of its own set: one or four multiply-adds a column and 128 inputs, where
// the plain layout takes sixteen.  More rows (awq_rows_kernel): a step is one set, the
// MFMA's rows are rows of x, and every step's sums are scaled.
//
// The waves of a workgroup take consecutive runs of sets of the same columns and
// add their sums through LDS in a fixed order; where the columns alone do not
// fill the card the sets are split over workgroups too, whose fp32 sums a
// second kernel adds.
#include "kernels.h"
#include "rows.h"

namespace moe {

namespace {

constexpr uint32_t kOutside = 0x80000000u;  // past the end of every buffer it is used with: the load gives 0

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
    int tiles;    // of columns
};

// The nibble that holds column c of a word: columns 0,2,4,6,1,3,5,7 lie in nibbles 0..7.
__device__ __forceinline__ int column_nibble(int c) { return c / 2 + 4 * (c % 2); }

__device__ __forceinline__ void put(const Awq& a, int64_t m, int n, float v) {
    if (a.f32) static_cast<float*>(a.y)[m * a.ldy + n] = v;
    else static_cast<uint16_t*>(a.y)[m * a.ldy + n] = (uint16_t)f32_to_bf16_bits(v);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ uint32_t load4(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t all) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, (int)lane, (int)all, 0);
}
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t all) {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)lane, (int)all, 0));
}

// The words of 8 inputs with their halves side by side: pair p holds inputs 2p and 2p + 1.
struct Halves {
    uint32_t lo[4], hi[4];
};
__device__ __forceinline__ Halves halves(const uint32_t* w, uint32_t select) {
    Halves v;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        v.lo[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], select);
        v.hi[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x07060302u);
    }
    return v;
}
// Masks and constants of the two conversions.  As literals they would cost an
// instruction each (v_and_or_b32 takes none), so a mask is kept in a vector and a
// constant in a scalar register, out of the compiler's sight.  The instruction
// itself is the compiler's: an MFMA has to wait two states for an operand that
// a vector instruction writes, and inside inline assembly it would not see that
// one does (and_or there gave wrong columns).
struct Bits {
    uint32_t mq, cq, mz, cz;
    __device__ __forceinline__ Bits() : mq(0x00780078u), cq(0x41804180u), mz(0x00780000u), cz(0x41800000u) {
        asm("" : "+v"(mq), "+v"(mz));
        asm("" : "+s"(cq), "+s"(cz));
    }
};

// 16 + q of nibble j, 8 inputs.
__device__ __forceinline__ bf16x8_t column(const Halves& v, int j, const Bits& k) {
    uint32_t b[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t h = j < 4 ? v.lo[p] : v.hi[p];
        b[p] = ((j % 4 == 0 ? h << 3 : h >> (4 * (j % 4) - 3)) & k.mq) | k.cq;
    }
    return __builtin_bit_cast(bf16x8_t, make_uint4(b[0], b[1], b[2], b[3]));
}
// 16 + z of nibble j.
__device__ __forceinline__ float zero_point(uint32_t z, int j, const Bits& k) {
    return __uint_as_float(((j < 5 ? z << (19 - 4 * j) : z >> (4 * j - 19)) & k.mz) | k.cz);
}
__device__ __forceinline__ f32x4_t mfma(u32x4_t x, bf16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x), b, c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8_t ones() {
    return __builtin_bit_cast(bf16x8_t, make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u));
}

// The sets [first, end) of a wave: whole groups.
struct Run {
    int first, end;
};
__device__ __forceinline__ Run run_of(const Awq& a, int wave, int waves) {
    // (at most 2^19 groups and 2^11 slices)
    const uint32_t groups = (uint32_t)a.K >> (5 + a.gshift), slices = gridDim.y * waves, slice = blockIdx.y * waves + wave;
    return {(int)(groups * slice / slices << a.gshift), (int)(groups * (slice + 1) / slices << a.gshift)};
}

// How the 16 lanes of a group share out a tile of 16 CW columns: with CW = 16
// a lane has two neighbouring words (and the 16 lanes read whole 128-byte
// lines), with 8 one word, with 4 or 2 a half or a byte of a word that two or
// four lanes read.  Tiles that share lines run on one XCD (its workgroups are
// every eighth), so that a line is fetched once; whole lines are spread over
// the XCDs (1 x 16384 x 16384: 32 us against 36).
template <int CW>
struct Lane {
    static constexpr int kW = CW > 8 ? CW / 8 : 1;      // words of a lane
    static constexpr int kShare = CW < 8 ? 8 / CW : 1;  // lanes of a word
    int tile;                                           // < 0: nothing to do
    int h;                                              // which part of the word
    uint32_t word;                                      // in a row of codes, within it
    uint32_t select;                                    // of v_perm: that part of two words, side by side
};
template <int CW>
__device__ __forceinline__ Lane<CW> lane_of(int n16, uint32_t n8, int tiles) {
    typedef Lane<CW> L;
    L l;
    int to = tiles;
    if (CW == 16) {
        l.tile = blockIdx.x;
    } else {
        const int xcd = blockIdx.x % 8, from = tiles * xcd / 8;  // (at most 2^19 tiles)
        to = tiles * (xcd + 1) / 8;
        l.tile = from + (int)(blockIdx.x / 8);
    }
    if (l.tile >= to) {
        l.tile = -1;
        return l;
    }
    l.h = n16 % L::kShare;
    const uint32_t w = (uint32_t)l.tile * 2 * CW + n16 * L::kW / L::kShare;
    l.word = w < n8 ? w : n8 - L::kW;  // lanes past the last word read it again; nothing of theirs is stored
    l.select = CW == 2 ? 0x0C040C00u + 0x00010001u * l.h : CW == 4 && l.h ? 0x07060302u : 0x05040100u;
    return l;
}
// Where column c of a tile lies: column j of lane n16.
struct Place {
    int j, n16;
};
template <int CW>
__device__ __forceinline__ Place place_of(int c) {
    const int nibble = column_nibble(c % 8), word = c / 8;
    if (CW >= 8) return {8 * (word % (CW / 8 ? CW / 8 : 1)) + nibble, word / (CW / 8 ? CW / 8 : 1)};
    return {nibble % CW, word * (8 / CW) + nibble / CW};
}

// W words of a lane (W neighbouring words of one row of codes).
template <int W>
struct Words {
    uint32_t v[W];
};
// Code rows: with two words a lane the 16 lanes read whole 128-byte lines, once
// (non-temporal); with one, two waves share a line through the cache.
template <int W>
__device__ __forceinline__ Words<W> load_words(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t all) {
    if constexpr (W == 2) {
        const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, (int)lane, (int)all, 2));
        return {{v.x, v.y}};
    } else {
        return {{load4(r, lane, all)}};
    }
}
// The scales of a lane's columns: of its words' 8 columns each, or (CW = 2) of
// the four columns among which its two lie.
template <int CW>
struct Scales {
    u32x4_t v[Lane<CW>::kW];
};
template <int CW>
__device__ __forceinline__ Scales<CW> load_scales(__amdgpu_buffer_rsrc_t r, uint32_t word, int h) {
    Scales<CW> s;
    if constexpr (CW == 2) {
        const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, (int)(16u * word + 8u * (h & 1)), 0, 0));
        s.v[0] = u32x4_t{v.x, v.y, 0, 0};
    } else {
#pragma unroll
        for (int i = 0; i < Lane<CW>::kW; ++i) s.v[i] = load16(r, 16u * word + 16u * i, 0);
    }
    return s;
}
// Nibble n of a word holds column 2 (n % 4) + n / 4.
template <int CW>
__device__ __forceinline__ float scale_of(const Scales<CW>& s, int j, int h) {
    const int half = CW == 2 ? h >> 1 : CW == 4 ? h : (j % 8) >> 2;
    return f16_to_f32((s.v[j / 8][CW == 2 ? j : j & 3] >> (16 * half)) & 0xFFFFu);
}
template <int W>
__device__ __forceinline__ Words<W> load_zeros(__amdgpu_buffer_rsrc_t r, uint32_t lane) {
    if constexpr (W == 2) {
        const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, (int)lane, 0, 0));
        return {{v.x, v.y}};
    } else {
        return {{load4(r, lane, 0)}};
    }
}

// Sum over the four groups of 16 lanes, in every lane.
__device__ __forceinline__ float sum_groups(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Up to MM rows (1 or 4).
template <int CW, int MM, int WV>
__global__ __launch_bounds__(64 * WV) void awq_few_kernel(Awq a) {
    typedef float rows_t __attribute__((ext_vector_type(MM)));
    constexpr int W = Lane<CW>::kW;
    __shared__ __align__(16) rows_t red[WV][CW][16];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int kq = lane / 16, n16 = lane % 16;
    const uint32_t n8 = a.N / 8;
    const Lane<CW> l = lane_of<CW>(n16, n8, a.tiles);
    if (l.tile < 0) return;
    const uint32_t wl = l.word;
    const int sets = a.K / 32;
    const Run r = run_of(a, wave, WV);

    uint32_t woff[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) woff[i] = 4u * ((32u * kq + i) * n8 + wl);
    const uint32_t goff = ((uint32_t)kq >> a.gshift) * n8 + wl;
    const uint32_t xoff = n16 / 4 == kq && n16 % 4 < a.M ? (uint32_t)(n16 % 4) * (uint32_t)a.ldx * 2 + 64u * kq : kOutside;

    // Steps 2h and 2h + 1 of four sets: 16 inputs of each set.  What lies behind
    // the last set is not read, nor is anything for sets past the run's end; a set
    // past the run's end beside others meets zeros of x.
    struct Half {
        u32x4_t x[2];
        Words<W> w[2][8];
    };
    auto fetch = [&](int set, int h, Half& f) {
        const int left = set >= r.end ? 0 : sets - set < 4 ? sets - set : 4;
        const int64_t at = set < r.end ? set : r.first;
        const __amdgpu_buffer_rsrc_t xb = buffer(a.x + at * 32, left ? (uint32_t)(a.M - 1) * (uint32_t)a.ldx * 2 + (uint32_t)left * 64u : 0u);
        const __amdgpu_buffer_rsrc_t q = buffer(a.qw + at * 32 * n8, (uint32_t)left * 128u * n8);
        const uint32_t xo = kq < r.end - set ? xoff : kOutside;
        // (an empty buffer's bound, which the scalar offset is taken from, stays 0)
        const uint32_t xstep = left ? 16u : 0u, wstep = left ? 32u * n8 : 0u;
#pragma unroll
        for (int u = 0; u < 2; ++u) f.x[u] = load16(xb, xo, xstep * (2 * h + u));
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) f.w[u][i] = load_words<W>(q, woff[i], wstep * (2 * h + u));
    };
    const f32x4_t none = f32x4_t(0.0f);
    const Bits bits;
    f32x4_t d[CW], sx;
    auto add = [&](const Half& f, bool begin) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            sx = mfma(f.x[u], ones(), begin && u == 0 ? none : sx);
#pragma unroll
            for (int v = 0; v < W; ++v) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = f.w[u][i].v[v];
                const Halves h = halves(w, l.select);
#pragma unroll
                for (int j = 0; j < CW / W; ++j) d[8 * v + j] = mfma(f.x[u], column(h, j, bits), begin && u == 0 ? none : d[8 * v + j]);
            }
        }
    };

    rows_t acc[CW];
#pragma unroll
    for (int j = 0; j < CW; ++j) acc[j] = rows_t(0.0f);
    if (r.first < r.end) {
        // half of the loads are always on their way: the order of loads and
        // products is kept
        Half f0, f1;
        fetch(r.first, 0, f0);
        for (int set = r.first; set < r.end; set += 4) {
            __builtin_amdgcn_sched_barrier(0);
            fetch(set, 1, f1);
            // (zeros and scales of the run's own groups only: its lanes past the end meet
            // scales of 0, as another run's infinity times their sum of 0 were NaN)
            const int left = r.end - set < 4 ? r.end - set : 4;
            const int g = set >> a.gshift, groups = (left + (1 << a.gshift) - 1) >> a.gshift;
            const Words<W> z = load_zeros<W>(buffer(a.qz + (int64_t)g * n8, (uint32_t)groups * 4u * n8), 4u * goff);
            const Scales<CW> s = load_scales<CW>(buffer(a.sc + (int64_t)g * n8 * 8, (uint32_t)groups * 16u * n8), goff, l.h);
            __builtin_amdgcn_sched_barrier(0);
            add(f0, true);
            __builtin_amdgcn_sched_barrier(0);
            fetch(set + 4, 0, f0);
            __builtin_amdgcn_sched_barrier(0);
            add(f1, false);
#pragma unroll
            for (int j = 0; j < CW; ++j) {
                const float zj = zero_point(z.v[j / 8] >> (CW < 8 ? 4 * CW * l.h : 0), j % 8, bits), sj = scale_of<CW>(s, j, l.h);
#pragma unroll
                for (int i = 0; i < MM; ++i) acc[j][i] = fmaf(sj, fmaf(-zj, sx[i], d[j][i]), acc[j][i]);
            }
        }
    }

#pragma unroll
    for (int j = 0; j < CW; ++j) {
        rows_t v;
#pragma unroll
        for (int i = 0; i < MM; ++i) v[i] = sum_groups(acc[j][i]);
        if (kq == 0) red[wave][j][n16] = v;
    }
    __syncthreads();
    // column c of the tile: the waves' sums, in order
    for (int c = threadIdx.x; c < 16 * CW; c += 64 * WV) {
        const int64_t n = (int64_t)l.tile * 16 * CW + c;
        const Place p = place_of<CW>(c);
        rows_t v = red[0][p.j][p.n16];
#pragma unroll
        for (int w = 1; w < WV; ++w) v += red[w][p.j][p.n16];
        if (n < a.N) {
#pragma unroll
            for (int i = 0; i < MM; ++i)
                if (i < a.M) {
                    if (a.part) a.part[((int64_t)blockIdx.y * a.M + i) * a.N + n] = v[i];
                    else put(a, i, (int)n, v[i]);
                }
        }
    }
}

// 16 MT rows.
template <int CW, int MT, int WV>
__global__ __launch_bounds__(64 * WV) void awq_rows_kernel(Awq a) {
    constexpr int W = Lane<CW>::kW, kPass = CW < 8 ? CW : 8;  // columns of a lane whose sums are added at a time
    __shared__ __align__(16) f32x4_t red[WV][kPass][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int kq = lane / 16, n16 = lane % 16;
    const uint32_t n8 = a.N / 8;
    const int m0 = blockIdx.z * 16 * MT;
    const Lane<CW> l = lane_of<CW>(n16, n8, a.tiles);
    if (l.tile < 0) return;
    const uint32_t wl = l.word;
    const Run r = run_of(a, wave, WV);

    uint32_t woff[8], xoff[MT];
#pragma unroll
    for (int i = 0; i < 8; ++i) woff[i] = 4u * ((8u * kq + i) * n8 + wl);
    const int rows = a.M - m0 < 16 * MT ? a.M - m0 : 16 * MT;
#pragma unroll
    for (int t = 0; t < MT; ++t) xoff[t] = 16 * t + n16 < rows ? (uint32_t)(16 * t + n16) * (uint32_t)a.ldx * 2 + 16u * kq : kOutside;
    const uint16_t* x0 = a.x + m0 * a.ldx;
    const uint32_t xbytes = (uint32_t)(rows - 1) * (uint32_t)a.ldx * 2 + 64u;

    struct Step {
        Words<W> z;
        Scales<CW> s;
        u32x4_t x[MT];
        Words<W> w[8];
    };
    auto fetch = [&](int set, Step& st) {
        const bool in = set < r.end;  // (past the run's end nothing is read)
        const int64_t at = in ? set : r.first, g = at >> a.gshift;
        const __amdgpu_buffer_rsrc_t q = buffer(a.qw + at * 32 * n8, in ? 128u * n8 : 0u);
        const __amdgpu_buffer_rsrc_t xb = buffer(x0 + at * 32, in ? xbytes : 0u);
#pragma unroll
        for (int t = 0; t < MT; ++t) st.x[t] = load16(xb, xoff[t], 0);
        st.z = load_zeros<W>(buffer(a.qz + g * n8, in ? 4u * n8 : 0u), 4u * wl);
        st.s = load_scales<CW>(buffer(a.sc + g * n8 * 8, in ? 16u * n8 : 0u), wl, l.h);
#pragma unroll
        for (int i = 0; i < 8; ++i) st.w[i] = load_words<W>(q, woff[i], 0);
    };
    f32x4_t acc[MT][CW];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < CW; ++j) acc[t][j] = f32x4_t(0.0f);
    const f32x4_t none = f32x4_t(0.0f);
    const Bits bits;
    auto add = [&](const Step& st) {
        f32x4_t sx[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) sx[t] = mfma(st.x[t], ones(), none);
        // a column's sums are used while the next column's are formed
        f32x4_t d[2][MT];
        Halves h;
#pragma unroll
        for (int j = 0; j <= CW; ++j) {
            if (j < CW) {
                if (j % 8 == 0) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = st.w[i].v[j / 8];
                    h = halves(w, l.select);
                }
                const bf16x8_t b = column(h, j % 8, bits);
#pragma unroll
                for (int t = 0; t < MT; ++t) d[j % 2][t] = mfma(st.x[t], b, none);
            }
            if (j > 0) {
                const int o = j - 1;
                const float zj = zero_point(st.z.v[o / 8] >> (CW < 8 ? 4 * CW * l.h : 0), o % 8, bits), sj = scale_of<CW>(st.s, o, l.h);
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][o][i] = fmaf(sj, fmaf(-zj, sx[t][i], d[o % 2][t][i]), acc[t][o][i]);
            }
        }
    };

    if (r.first < r.end) {
        // the next step's loads are on their way while one is added: the order of
        // loads and products is kept
        Step s0, s1;
        fetch(r.first, s0);
        for (int s = r.first; s < r.end; s += 2) {
            __builtin_amdgcn_sched_barrier(0);
            fetch(s + 1, s1);
            __builtin_amdgcn_sched_barrier(0);
            add(s0);
            __builtin_amdgcn_sched_barrier(0);
            fetch(s + 2, s0);
            __builtin_amdgcn_sched_barrier(0);
            if (s + 1 < r.end) add(s1);
        }
    }

    // the waves' sums, 16 rows and up to 8 columns of each lane at a time: thread
    // (row quad, c) adds four rows of column c
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int v = 0; v < W; ++v) {
            if (t || v) __syncthreads();
#pragma unroll
            for (int j = 0; j < kPass; ++j) red[wave][j][lane] = acc[t][kPass * v + j];
            __syncthreads();
            for (int o = threadIdx.x; o < 64 * kPass; o += 64 * WV) {
                const int c = o % (16 * kPass), quad = o / (16 * kPass);
                const Place p = place_of<kPass>(c);
                f32x4_t sum = red[0][p.j][16 * quad + p.n16];
#pragma unroll
                for (int w = 1; w < WV; ++w) sum += red[w][p.j][16 * quad + p.n16];
                const int64_t n = (int64_t)l.tile * 16 * CW + (W > 1 ? (c / 8 * W + v) * 8 + c % 8 : c);
                if (n < a.N) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int64_t m = m0 + 16 * t + 4 * quad + i;
                        if (m < a.M) {
                            if (a.part) a.part[((int64_t)blockIdx.y * a.M + m) * a.N + n] = sum[i];
                            else put(a, m, (int)n, sum[i]);
                        }
                    }
                }
            }
        }
}

// y = the `splits` partial sums, in order; a row of y a grid row.
__global__ __launch_bounds__(256) void awq_sum_kernel(Awq a, int splits) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= a.N) return;
    const int64_t m = blockIdx.y, one = (int64_t)a.M * a.N;
    const float* part = a.part + m * a.N + n;
    float v = 0.0f;
    for (int s = 0; s < splits; s += 8) {
        float p[8];  // eight loads on their way at a time
#pragma unroll
        for (int u = 0; u < 8; ++u) p[u] = part[(s + u < splits ? s + u : s) * one];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (s + u < splits) v += p[u];
    }
    put(a, m, n, v);
}

// How a call is cut up.  Measured (one, 13 or 16 rows; us, sum kernel included):
//   columns of a lane: whole lines matter to large matrices, workgroups to small ones:
//     8192 x 8192: 16 columns 12.9, 8 14.5, 4 18.5, 2 24; 2560 x 2560: 16 8.4, 8 6.9 (split) 8.9 (not), 2 6.3;
//     16384 columns x 1280 inputs: 8 7.0, 4 5.9, 2 7.9.  16 need N % 16 == 0 for aligned pairs of words.
//   splits: workgroups for every compute unit (8192 x 8192: 1 37, 4 15.9, 8 12.9, 16 14.7), but inputs up to 4096 deep
//     are not split, which would save up to 2 us of kernel and cost a launch (4096 x 4096: 9.2, split 7.3).
//   waves: 4; the large matrices of more than four rows 8 (16 x 16384 x 16384: 36 against 39).
struct Plan {
    int cw, mt, waves, tiles, splits, rows;  // mt = 0: up to four rows
};

Plan plan(int M, int N, int K, bool pairs) {
    Plan p;
    p.mt = M <= 4 ? 0 : M <= 16 ? 1 : 2;
    p.rows = p.mt ? (M + 16 * p.mt - 1) / (16 * p.mt) : 1;
    const bool large = (int64_t)N * K >= (1 << 25), split = large || K > 4096;
    if (large) p.cw = pairs ? 16 : 8;
    else if (split) p.cw = 4;
    else p.cw = N <= 8192 ? 2 : N <= 16384 ? 4 : 8;
    p.waves = large && p.mt ? 8 : 4;
    p.tiles = (N + 16 * p.cw - 1) / (16 * p.cw);
    const int64_t fill = 256 / ((int64_t)p.tiles * p.rows);
    const int64_t deep = K / 32 / (p.waves * (large ? 4 : 8));  // sets a wave takes at least
    const int64_t s = fill < deep ? fill : deep;
    p.splits = split && s > 1 ? (int)s : 1;
    return p;
}

template <int CW, int WV>
void run_awq_rows(const Awq& a, const Plan& p, hipStream_t s) {
    const dim3 grid((p.tiles + 7) / 8 * 8, p.splits, p.rows), block(64 * WV);
    if (p.mt == 2) hipLaunchKernelGGL((awq_rows_kernel<CW, 2, WV>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((awq_rows_kernel<CW, 1, WV>), grid, block, 0, s, a);
}
template <int CW>
void run_awq_few(const Awq& a, const Plan& p, hipStream_t s) {
    const dim3 grid((p.tiles + 7) / 8 * 8, p.splits, 1), block(64 * 4);
    if (a.M == 1) hipLaunchKernelGGL((awq_few_kernel<CW, 1, 4>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((awq_few_kernel<CW, 4, 4>), grid, block, 0, s, a);
}

}  // namespace

// Bytes of the partial sums of M rows.
static size_t part_bytes(int M, int N, int K) {
    // whether pairs of words are aligned is known with the pointers only
    const int s = plan(M, N, K, N % 16 == 0).splits, t = plan(M, N, K, false).splits;
    const int most = s > t ? s : t;
    return most > 1 ? (size_t)most * M * N * sizeof(float) : 0;
}

size_t awq_matmul_ws_bytes(int M, int N, int K) {
    // the most that any smaller M needs: the splits fall where M takes another kernel or row of tiles
    size_t most = part_bytes(M, N, K);
    const int tops[2] = {4, 16};
    for (int m : tops)
        if (m < M && part_bytes(m, N, K) > most) most = part_bytes(m, N, K);
    for (int m = 32; m < M && m <= 32 * 256; m += 32)  // (256 workgroups are never split)
        if (part_bytes(m, N, K) > most) most = part_bytes(m, N, K);
    return most;
}

size_t awq_matmul_needs(int M, int N, int K) { return part_bytes(M, N, K); }

hipError_t launch_awq_matmul(const uint16_t* x, int64_t ldx, const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                             int M, int N, int K, int group, int out_f32, void* y, int64_t ldy, void* ws, hipStream_t s) {
    Awq a{};
    a.x = x; a.ldx = ldx;
    a.qw = reinterpret_cast<const uint32_t*>(qweight);
    a.qz = reinterpret_cast<const uint32_t*>(qzeros);
    a.sc = scales;
    a.M = M; a.N = N; a.K = K; a.gshift = group == 32 ? 0 : group == 64 ? 1 : 2;
    a.f32 = out_f32; a.y = y; a.ldy = ldy;
    const Plan p = plan(M, N, K, N % 16 == 0 && ((uintptr_t)qweight | (uintptr_t)qzeros) % 8 == 0);
    a.part = p.splits > 1 ? static_cast<float*>(ws) : nullptr;
    a.tiles = p.tiles;
    if (!p.mt) {  // (four waves)
        if (p.cw == 16) run_awq_few<16>(a, p, s);
        else if (p.cw == 8) run_awq_few<8>(a, p, s);
        else if (p.cw == 4) run_awq_few<4>(a, p, s);
        else run_awq_few<2>(a, p, s);
    } else if (p.waves == 8) {  // (large matrices)
        if (p.cw == 16) run_awq_rows<16, 8>(a, p, s);
        else run_awq_rows<8, 8>(a, p, s);
    } else {
        if (p.cw == 8) run_awq_rows<8, 4>(a, p, s);
        else if (p.cw == 4) run_awq_rows<4, 4>(a, p, s);
        else run_awq_rows<2, 4>(a, p, s);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL(awq_sum_kernel, dim3((N + 255) / 256, M), dim3(256), 0, s, a, p.splits);  // (split: at most 128 x 32 rows)
    return hipGetLastError();
}

}  // namespace moe
