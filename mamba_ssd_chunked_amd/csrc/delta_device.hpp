// Device-side building blocks of the gated delta rule (gfx950, wave64).
//
// Every product runs on the bf16 matrix cores (16x16x32).  An fp32 operand is cut into
// three bf16 parts, each the rounded remainder of the ones before it, which together
// hold all 24 bits; a bf16 input is one part.  A product of an a-part and a b-part
// operand sums the pairs whose combined weight reaches fp32's last bit: 1 x 3 parts take
// three MFMAs, 3 x 3 six, and accumulate in fp32.  (An fp32 MFMA takes the time of about
// sixteen bf16 ones for the same product: v_mfma_f32_16x16x4_f32 issues in 32 cycles for
// k = 4, v_mfma_f32_16x16x32_bf16 in 16 for k = 32.)
//
// Operand and result layout of the 16x16x32 MFMA, for lane L (i = L % 16, g = L / 16):
// operands hold row / column i and eight k values, results hold D[4g + v][i], v = 0..3.
// Which k a slot means is free as long as both operands agree, so two results stacked
// along their row axis serve as the next product's operand without moving between lanes:
// slots 0..3 are rows 4g..4g+3 of the even tile, slots 4..7 of the odd one.
#pragma once

#include "ssd_device.hpp"

namespace ssd {

constexpr int DL = 64;         // tokens per chunk of the delta rule
constexpr int DTRI = 6;        // 16 x 32 operand tiles of a triangular 64 x 64 matrix
constexpr int DTILE = 64 * 8;  // bf16 values of one operand tile (8 per lane)

// Floats of a chunk's coefficients: e^G (zero past the row's length), e^{G_L - G}, beta, and
// e^{G_L} in the first of the next 64; then G in base 2 (fp64).
constexpr int DCF = 4 * DL;
constexpr int DCOEF = DCF + 2 * DL;

// Buffers of the scans, typed.
template <class T>
struct DeltaScan {
    const T *q, *k, *v, *dy;
    T* y;
    const int64_t* len;
    const float *init, *d_final;
    float *final_state, *d_init;
    float* coef;
    uint16_t *M, *P, *NT;
    float *H, *E, *dH, *dZ, *carry;
    int segs, seg_chunks;  // segments of the chunk axis, and their chunks
};

// A vector from memory on 16 bytes, as the entry points ask for (the type of eight floats alone says 32).
template <class V>
__device__ __forceinline__ V load_vec(const void* at) {
    typedef V there __attribute__((aligned(16)));
    return *static_cast<const there*>(at);
}

template <int N>
struct Parts {
    b8v p[N];
};

// Eight fp32 values as N bf16 parts, each rounded to nearest even.
template <int N>
__device__ __forceinline__ Parts<N> split8(const float (&x)[8]) {
    Parts<N> o;
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = f32x2_to_bf16x2(r[2 * e], r[2 * e + 1]);
            if (n + 1 < N) {
                r[2 * e] -= __uint_as_float(w[e] << 16);
                r[2 * e + 1] -= __uint_as_float(w[e] & 0xffff0000u);
            }
        }
        o.p[n] = __builtin_bit_cast(b8v, *reinterpret_cast<const uint4*>(w));
    }
    return o;
}
template <int N>
__device__ __forceinline__ Parts<N> split44(v4f a, v4f b) {
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return split8<N>(x);
}

// The same for T results at once, the MFMAs of one result T apart: a dependent MFMA waits for
// its accumulator.
template <int NA, int NB, int T>
__device__ __forceinline__ void mma_a(v4f (&c)[T], const Parts<NA> (&a)[T], const Parts<NB>& b) {
    constexpr int K = (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int s = K; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t].p[i], b.p[s - i], c[t], 0, 0, 0);
}
template <int NA, int NB, int T>
__device__ __forceinline__ void mma_b(v4f (&c)[T], const Parts<NA>& a, const Parts<NB> (&b)[T]) {
    constexpr int K = (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int s = K; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b[t].p[s - i], c[t], 0, 0, 0);
}

template <int NA, int NB>
__device__ __forceinline__ v4f mma(const Parts<NA>& a, const Parts<NB>& b, v4f c) {
    constexpr int K = (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int s = K; s >= 0; --s)  // the small terms first
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[s - i], c, 0, 0, 0);
    return c;
}

// The result of a 16x16x32 MFMA may be read by other instructions eight wait states after its
// issue; the compiler counts them inside a loop body but not across its back edge (clang 22 of
// ROCm 7.2 read an accumulator two states after the last MFMA of the iteration before: wrong
// values in the registers written last).  To stand at the end of a loop body that carries
// accumulators.
__device__ __forceinline__ void mfma_settle() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 3" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Four bf16 of one column out of a row-major LDS matrix: the 16 lanes of a group address
// four rows x 16 columns, 8 bytes each (lane i: row i / 4, columns 4 (i % 4) .. + 3), and
// lane i receives column i of the four rows.
typedef s4 __attribute__((address_space(3))) lds_s4;
__device__ __forceinline__ s4 lds_col4(const uint16_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
}
__device__ __forceinline__ b8v join8(s4 a, s4 b) {
    typedef short s8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(b8v, s8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

// 16 bytes per lane from global memory straight into LDS at lds + 16 lane (a byte address, the
// same in all lanes).  It counts in vmcnt; the reader waits and passes a barrier
// (wait_barrier).  Written out because around the builtin the compiler waits for every such
// load before any LDS read, of whatever array.  m0, which holds the address, is the compiler's: a
// clobber list cannot give it away, so it is put back.
typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char*)p));
}
__device__ __forceinline__ void load_to_lds(const void* src, uint32_t lds) {
    uint32_t was;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(was)
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
                 : "memory");
}
// Wait until at most N of this wave's memory operations are outstanding (they end in order) and
// its LDS reads have returned, then for the workgroup.
template <int N>
__device__ __forceinline__ void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N < 63 ? N : 63) : "memory");
}

// Sum over N = 4, 8, 16 or 32 consecutive lanes, in all of them: inside a row of sixteen by the
// vector unit's own lane moves (mirrored halves, then swaps in pairs; rotations of a whole row).
template <int CTRL>
__device__ __forceinline__ float moved(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int N>
__device__ __forceinline__ float sum_over_lanes(float x) {
    static_assert(N == 4 || N == 8 || N == 16 || N == 32);
    if constexpr (N >= 16) {
        x += moved<0x128>(x);
        x += moved<0x124>(x);
        x += moved<0x122>(x);
        x += moved<0x121>(x);
        if constexpr (N == 32) x += __shfl_xor(x, 16);
    } else {
        if constexpr (N == 8) x += moved<0x141>(x);  // lane 7 - i
        x += moved<0x4e>(x);                         // lane i ^ 2
        x += moved<0xb1>(x);                         // lane i ^ 1
    }
    return x;
}

// LDS order of a 64-token matrix [64, r] of bf16: 16 x 32 tiles (token tile tau, step j), each
// a kilobyte: the eight values r = 32 j + 8 g .. of token 16 tau + i at 16-byte slot
// 16 g + (i ^ 4 g).  A tile is then one lane-linear operand read (rows), and the four rows x four
// column groups that a transposing read (columns) addresses lie in sixteen different slots mod 16.
__device__ __forceinline__ constexpr int tile_slot(int i, int g) { return 16 * g + (i ^ (4 * g)); }

// Operand tile numbers of a lower (upper) triangular 64 x 64 matrix in row tiles tau of 16
// and k steps j of 32: the six tiles that are not zero.
__device__ __forceinline__ constexpr int tri_lower(int tau, int j) { return tau < 2 ? tau : 2 * (tau - 1) + j; }
__device__ __forceinline__ constexpr int tri_upper(int tau, int j) { return tau < 2 ? 2 * tau + j : tau + 2; }

// Parts of a value of the io type.
template <class IO>
__host__ __device__ constexpr int in_parts() { return sizeof(typename IO::T) == 2 ? 1 : 3; }

// Eight io values as bf16 parts, zeros where !on.
template <class IO, class V>
__device__ __forceinline__ Parts<in_parts<IO>()> parts_of(const V& x, bool on) {
    Parts<in_parts<IO>()> o;
    if constexpr (in_parts<IO>() == 1) {
        uint4 w = __builtin_bit_cast(uint4, x);
        if (!on) w = make_uint4(0, 0, 0, 0);
        o.p[0] = __builtin_bit_cast(b8v, w);
    } else {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = on ? x[e] : 0.0f;
        o = split8<3>(f);
    }
    return o;
}
}  // namespace ssd
