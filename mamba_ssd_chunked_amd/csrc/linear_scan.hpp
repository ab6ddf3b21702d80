// The scan over chunks that every part of linear attention runs (k_linear.hip states the mathematics).
#pragma once

#include <type_traits>

#include "delta_device.hpp"
#include "linear_power.hpp"
#include "ssd_launch.hpp"

namespace ssd {

constexpr int LC = 32;  // tokens per chunk

// The eight XCDs take workgroups in turn and each has its own L2: give each a consecutive run of
// the work, so that the columns, value heads and gradients that read the same rows meet in one.
__device__ __forceinline__ int64_t linear_order(int64_t blk, int64_t n) {
    const int64_t x = blk % 8, q = n / 8, rem = n % 8;
    return x * q + (x < rem ? x : rem) + blk / 8;
}

// kWide: outputs in fp32 whatever the io type.
enum LinMode { kOutputs, kWide, kCarry, kTangent, kTangentCarry };

// Eight fp32 values as N bf16 parts like split8, the remainders by two-term dot products with (-1, 0) and
// (0, -1): exact, and without taking the parts out of their words first (seven instructions a pair instead
// of eleven).  The first of the two constants has to come from a register: as an immediate the
// instruction takes it for both terms.
template <int N>
__device__ __forceinline__ Parts<N> cut8(const float (&x)[8]) {
    uint32_t first = 0x0000bf80u;
    asm("" : "+s"(first));
    const v2bf lo = __builtin_bit_cast(v2bf, first), hi = __builtin_bit_cast(v2bf, 0xbf800000u);
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
                r[2 * e] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, w[e]), lo, r[2 * e], false);
                r[2 * e + 1] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, w[e]), hi, r[2 * e + 1], false);
            }
        }
        o.p[n] = __builtin_bit_cast(b8v, *reinterpret_cast<const uint4*>(w));
    }
    return o;
}
template <int N>
__device__ __forceinline__ Parts<N> cut44(v4f a, v4f b) {
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return cut8<N>(x);
}

// One workgroup: NW waves with NTILE tiles of 16 value columns each of one head, through the chunks of a
// segment.  A wave keeps its columns' state in registers.  A chunk's rows are fetched into registers while
// the chunk before is worked on, and lie in LDS as operand tiles: a barrier before they are read, one
// after the causal matrix P is, and one when all is read.
//
// What bounds it: the bytes of the rows and the LDS reads of the operands, about as much time each, and the
// two overlap by half (512 heads of 4096 tokens, p = 64, r = 128, bf16: loads and stores alone 352 us, the
// rest alone 363, together 440; P, q H^T, P V and the state take 43, 72, 39 and 77 of them).
template <class IO, int R, int NTILE, int NW, int MODE>
struct LinearScan {
    using T = typename IO::T;
    static constexpr int THREADS = 64 * NW;
    static constexpr int C = LC, NP = in_parts<IO>(), TT = C / 16;
    static constexpr int RP = R < 32 ? 32 : R, KJ = RP / 32, RT = RP / 16;
    static constexpr int PC = 16 * NTILE * NW, VJ = (PC + 31) / 32;
    static constexpr bool PLAIN = MODE == kOutputs || MODE == kWide, OUT = PLAIN || MODE == kTangent;
    static constexpr bool TAN = MODE == kTangent || MODE == kTangentCarry;
    using Out = typename std::conditional<MODE == kWide, float, T>::type;
    static constexpr int GT = TAN && NP > 1 ? 1 : 2;  // state tiles at a time (more in parts spill beside two states)
    static constexpr int QT = TT * KJ;  // operand tiles of q or k, a part
    static constexpr int VS = PC + 4;   // floats of a row of v (fp32 io)
    static constexpr int QBYTES = NP * QT * 1024, VBYTES = NP == 1 ? TT * VJ * 1024 : C * VS * 4;
    static constexpr int PBYTES = PLAIN ? 3 * TT * 1024 : MODE == kTangent ? VBYTES : 0;  // (P, or dy like v)
    static constexpr int YS = PC * sizeof(Out) + 16;  // bytes of a row of outputs
    static constexpr int oK = 0, oQ = oK + QBYTES, oV = oQ + (OUT ? QBYTES : 0), oP = oV + VBYTES, oY = oP + PBYTES,
                         oF = oY + (PLAIN ? C * YS : 0), LDS = oF + 4 * (MODE == kTangent ? 4 : 2) * C;
    // loads of one wave and of one thread
    static constexpr int PER = (QT + NW - 1) / NW;
    static constexpr int RPP = 16 / NTILE;  // rows of v that the workgroup loads at a time (fp32 io)
    static constexpr int VPER = NP == 1 ? (TT * VJ + NW - 1) / NW : C / RPP;
    typedef T raw8 __attribute__((ext_vector_type(8)));
    typedef T raw4 __attribute__((ext_vector_type(4)));
    using rawv = typename std::conditional<NP == 1, raw8, raw4>::type;
    typedef v4f State[NTILE][RT];

    char* sm;
    const LinearShape d;  // by value: through references the kernel's arguments are read again in every chunk
    const LinearJob a;
    // what a token's key adds to the state is scaled by, and to the tangent; what a token's query reads of the
    // tangent and of the state (kTangent)
    float *kf, *kft, *qw, *qwt;
    // scaled a^(t - s) of a lane's places t = i, s = 4 g + v in a tile of P on the diagonal (0 above it)
    // and in the one below
    v4f near, next;
    int lane, w, i, g, p0, wc, seg, h, b, len, chunks, c0, c1;
    int64_t bh, size;
    bool active;
    double l2;

    // The segment's columns p0 .. of head bh = (b, h).
    __device__ LinearScan(char* smem, const LinearShape& dd, const LinearJob& aa, int64_t head_, int segment, int first)
        : sm(smem), d(dd), a(aa), p0(first), seg(segment), bh(head_) {
        kf = reinterpret_cast<float*>(sm + oF);
        kft = kf + C;
        qw = kf + 2 * C;
        qwt = kf + 3 * C;
        lane = threadIdx.x & 63;
        w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        i = lane & 15;
        g = lane >> 4;
        h = static_cast<int>(bh % d.H);
        b = static_cast<int>(bh / d.H);
        len = d.len ? static_cast<int>(d.len[b]) : d.S;
        chunks = (len + C - 1) / C;
        c0 = seg * d.seg_chunks < chunks ? seg * d.seg_chunks : chunks;
        c1 = c0 + d.seg_chunks < chunks ? c0 + d.seg_chunks : chunks;
        l2 = log2_decay(d.log_decay[h]);
        wc = w * 16 * NTILE;  // this wave's first column, in the workgroup
        active = p0 + wc < d.P;
        size = static_cast<int64_t>(d.P) * R;
    }

    // ---------------------------------------------------------------- state
    // s[e][rho][v]: row r = 32 (rho / 2) + 8 g + 4 (rho % 2) + v, column col_of(i, e)
    // column of row / operand lane m of column tile e, from the wave's first
    __device__ static int col_of(int m, int e) { return NTILE == 1 ? m : 8 * (m >> 2) + 4 * e + (m & 3); }
    __device__ int row_of(int rho) const { return 32 * (rho >> 1) + 8 * g + 4 * (rho & 1); }
    template <class F>
    __device__ void each_state(F&& f) const {  // f(e, rho, column, row)
#pragma unroll
        for (int e = 0; e < NTILE; ++e)
#pragma unroll
            for (int rho = 0; rho < RT; ++rho)
                if (R >= 32 || row_of(rho) < R) f(e, rho, p0 + wc + col_of(i, e), row_of(rho));
    }
    __device__ void load_state(State& x, const float* src, int64_t sc, int64_t sr) const {
#pragma unroll
        for (int e = 0; e < NTILE; ++e)
#pragma unroll
            for (int rho = 0; rho < RT; ++rho) x[e][rho] = zero4();
        if (!src || !active) return;
        if (sr == 1)
            each_state([&](int e, int rho, int col, int row) { x[e][rho] = *reinterpret_cast<const v4f*>(src + col * sc + row); });
        else
            each_state([&](int e, int rho, int col, int row) {
#pragma unroll
                for (int v = 0; v < 4; ++v) x[e][rho][v] = src[col * sc + (row + v) * sr];
            });
    }
    __device__ void store_state(const State& x, float* dst, int64_t sc, int64_t sr) const {
        if (!dst || !active) return;
        if (sr == 1)
            each_state([&](int e, int rho, int col, int row) { *reinterpret_cast<v4f*>(dst + col * sc + row) = x[e][rho]; });
        else
            each_state([&](int e, int rho, int col, int row) {
#pragma unroll
                for (int v = 0; v < 4; ++v) dst[col * sc + (row + v) * sr] = x[e][rho][v];
            });
    }

    // ---------------------------------------------------------------- loads, a chunk ahead
    struct Ahead {
        raw8 k[PER], q[OUT ? PER : 1];
        rawv v[VPER], dy[MODE == kTangent ? VPER : 1];
    };
    __device__ int64_t token(int u) const {  // of place u of the row; past its end the last one
        u = u < len ? u : len - 1;
        return a.rev ? len - 1 - u : u;
    }
    // Place and columns of an operand tile that a lane loads: four neighbouring lanes have 64 bytes of a row
    // (bf16), where the address unit takes them at a time; with neighbours in neighbouring rows it took
    // four times as long, longer than anything else in a chunk.  Their slots in LDS lie in different banks.
    __device__ int slot_token() const { return lane >> 2; }
    __device__ int slot_at() const { return tile_slot(lane >> 2, lane & 3) * 16; }
    __device__ const T* head(const void* x, const int64_t (&stride)[3], int div) const {
        return static_cast<const T*>(x) + b * stride[0] + (h / div) * stride[2];
    }
    // Addresses of 16 places (a tile's) of a chunk: a pointer all lanes share and a 32-bit offset of the
    // lane's own, which is the same in every whole chunk; in the last one's, which stop at the row's end,
    // the pointer is the chunk's.
    __device__ bool whole(int c) const { return (c + 1) * C <= len; }
    __device__ int64_t first_row(int c) const { return !a.rev ? c * C : whole(c) ? len - (c + 1) * C : 0; }
    __device__ uint32_t shared_row(int c, int at, int rows) const { return !whole(c) ? 0 : a.rev ? C - rows - at : at; }
    __device__ uint32_t own_row(int u, int rows) const { return a.rev ? rows - 1 - u : u; }  // of a whole chunk
    __device__ uint32_t row_clamped(int c, int u) const { return static_cast<uint32_t>(token(c * C + u) - first_row(c)); }
    __device__ void fetch(Ahead& x, int c) const {
        const int64_t r0 = first_row(c);
        auto base = [&](const void* from, const int64_t(&stride)[3], int div) {
            return reinterpret_cast<const char*>(head(from, stride, div) + r0 * stride[1]);
        };
        const char *kp = base(a.k, a.ks, a.kdiv), *qp = base(a.q, a.qs, a.qdiv), *vp = base(a.v, a.vs, a.vdiv) + p0 * sizeof(T);
        const char* dp = MODE == kTangent ? base(a.dst, a.os, 1) + p0 * sizeof(T) : nullptr;
        const uint32_t kt = a.ks[1] * sizeof(T), qt = a.qs[1] * sizeof(T), vt = a.vs[1] * sizeof(T),
                       dt = a.os[1] * sizeof(T);
        const int is = slot_token();
        const uint32_t col = (8 * (lane & 3) < R ? 8 * (lane & 3) : 0) * sizeof(T);
        auto load = [](const char* at, uint32_t off, auto& to) {
            to = load_vec<std::remove_reference_t<decltype(to)>>(at + off);
        };
        uint32_t kr[PER], vr[VPER];  // rows
        const int vrow = NP == 1 ? is : threadIdx.x / (PC / 4);
        constexpr int VROWS = NP == 1 ? 16 : RPP;
        auto k_at = [&](int m) { return 16 * ((w + NW * m) / KJ); };
        auto v_at = [&](int m) { return NP == 1 ? 16 * ((w + NW * m) / VJ) : RPP * m; };
#pragma unroll
        for (int m = 0; m < PER; ++m) kr[m] = own_row(is, 16);
#pragma unroll
        for (int m = 0; m < VPER; ++m) vr[m] = own_row(vrow, VROWS);
        if (!whole(c)) {
#pragma unroll
            for (int m = 0; m < PER; ++m) kr[m] = row_clamped(c, k_at(m) + is);
#pragma unroll
            for (int m = 0; m < VPER; ++m) vr[m] = row_clamped(c, v_at(m) + vrow);
        }
#pragma unroll
        for (int m = 0; m < PER; ++m)
            if (QT % NW == 0 || w + NW * m < QT) {
                const uint32_t row = shared_row(c, k_at(m), 16), j = 32 * ((w + NW * m) % KJ) * sizeof(T);
                load(kp + row * kt + j, kr[m] * kt + col, x.k[m]);
                if constexpr (OUT) load(qp + row * qt + j, kr[m] * qt + col, x.q[m]);
            }
#pragma unroll
        for (int m = 0; m < VPER; ++m)
            if (NP != 1 || TT * VJ % NW == 0 || w + NW * m < TT * VJ) {
                const int vcol = p0 + (NP == 1 ? 32 * ((w + NW * m) % VJ) + 8 * (lane & 3) : 4 * (threadIdx.x % (PC / 4)));
                const uint32_t to = (vcol < d.P ? vcol - p0 : 0) * sizeof(T), row = shared_row(c, v_at(m), VROWS);
                load(vp + row * vt, vr[m] * vt + to, x.v[m]);
                if constexpr (MODE == kTangent) load(dp + row * dt, vr[m] * dt + to, x.dy[m]);
            }
    }
    __device__ static Parts<NP> parts8(const raw8& x) {
        if constexpr (NP == 1) {
            Parts<NP> o;
            o.p[0] = __builtin_bit_cast(b8v, x);
            return o;
        } else {
            const float f[8] = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
            return cut8<NP>(f);
        }
    }
    // Into LDS, tokens from n on as zeros.
    __device__ void put(Ahead& x, int n) const {
        const int is = slot_token();
        const bool part = n < C;
        auto blank = [](auto& r, bool on) {
#pragma unroll
            for (int e = 0; e < static_cast<int>(sizeof(r) / sizeof(T)); ++e) r[e] = on ? r[e] : T(0);
        };
#pragma unroll
        for (int m = 0; m < PER; ++m) {
            const int tile = w + NW * m, tau = tile / KJ;
            if (QT % NW == 0 || tile < QT) {
                if (R < 32 || part) {
                    const bool on = 16 * tau + is < n && (R >= 32 || 8 * (lane & 3) < R);
                    blank(x.k[m], on);
                    if constexpr (OUT) blank(x.q[m], on);
                }
                const auto kx = parts8(x.k[m]);
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    *reinterpret_cast<b8v*>(sm + oK + (q * QT + tile) * 1024 + slot_at()) = kx.p[q];
                if constexpr (OUT) {
                    const auto qx = parts8(x.q[m]);
#pragma unroll
                    for (int q = 0; q < NP; ++q)
                        *reinterpret_cast<b8v*>(sm + oQ + (q * QT + tile) * 1024 + slot_at()) = qx.p[q];
                }
            }
        }
        put_values(x.v, oV, n);
        if constexpr (MODE == kTangent) put_values(x.dy, oP, n);
    }
    __device__ void put_values(rawv (&x)[VPER], int base, int n) const {
        auto blank = [](auto& r, bool on) {
#pragma unroll
            for (int e = 0; e < static_cast<int>(sizeof(r) / sizeof(T)); ++e) r[e] = on ? r[e] : T(0);
        };
#pragma unroll
        for (int m = 0; m < VPER; ++m) {
            if constexpr (NP == 1) {
                const int tile = w + NW * m, tau = tile / VJ;
                if (TT * VJ % NW == 0 || tile < TT * VJ) {
                    if (n < C) blank(x[m], 16 * tau + slot_token() < n);
                    *reinterpret_cast<raw8*>(sm + base + tile * 1024 + slot_at()) = x[m];
                }
            } else {
                const int row = RPP * m + threadIdx.x / (PC / 4);
                if (n < C) blank(x[m], row < n);
                *reinterpret_cast<raw4*>(sm + base + (row * VS + 4 * (threadIdx.x % (PC / 4))) * 4) = x[m];
            }
        }
    }
    // powers by which the tokens of a chunk of n reach its end
    __device__ void put_factors(int n) const {
        if (threadIdx.x < C) {
            const int e = n - 1 - static_cast<int>(threadIdx.x);
            const float f = e >= 0 ? a.in * power(l2, e + a.rev) : 0.0f;
            kf[threadIdx.x] = f;
            if constexpr (TAN) kft[threadIdx.x] = static_cast<float>(e) * f;
        }
    }

    // ---------------------------------------------------------------- operands
    __device__ Parts<NP> row_op(int base, int tau, int j) const {  // rows: tokens 16 tau + i
        Parts<NP> o;
#pragma unroll
        for (int n = 0; n < NP; ++n)
            o.p[n] = *reinterpret_cast<const b8v*>(sm + base + (n * QT + tau * KJ + j) * 1024 + tile_slot(i, g) * 16);
        return o;
    }
    __device__ Parts<NP> col_op(int rho, int base = oK) const {  // rows of state tile rho, k over the chunk's tokens
        Parts<NP> o;
        const int at = base + (rho >> 1) * 1024 + tile_slot(4 * g + (i >> 2), i & 3) * 16 + (rho & 1) * 8;
#pragma unroll
        for (int n = 0; n < NP; ++n)
            o.p[n] = join8(lds_col4(reinterpret_cast<const uint16_t*>(sm + at + n * QT * 1024)),
                           lds_col4(reinterpret_cast<const uint16_t*>(sm + at + (n * QT + KJ) * 1024)));
        return o;
    }
    // tokens 16 t + 4 g + v of column col_of(i, e), as they lie (bf16) or as values (fp32)
    __device__ auto value4(int t, int e, int base = oV) const {
        if constexpr (NP == 1) {
            const int col = wc + (NTILE == 1 ? 4 * (i & 3) : 8 * (i & 3) + 4 * e);
            return lds_col4(reinterpret_cast<const uint16_t*>(
                sm + base + (t * VJ + (col >> 5)) * 1024 + tile_slot(4 * g + (i >> 2), (col >> 3) & 3) * 16 +
                ((col >> 2) & 1) * 8));
        } else {
            const float* x = reinterpret_cast<const float*>(sm + base) + (16 * t + 4 * g) * VS + wc + col_of(i, e);
            return v4f{x[0], x[VS], x[2 * VS], x[3 * VS]};
        }
    }
    // all 32 tokens of column col_of(i, e), times what each is weighted by
    __device__ void values(v4f (&val)[2], int e, int base = oV) const {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const auto x = value4(t, e, base);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if constexpr (NP == 1)
                    val[t][m] = bf16_to_f32(x[m]);
                else
                    val[t][m] = x[m];
            }
        }
    }
    __device__ Parts<3> weighted(const v4f (&val)[2], const float* by) const {
        return cut44<3>(val[0] * *reinterpret_cast<const v4f*>(by + 4 * g), val[1] * *reinterpret_cast<const v4f*>(by + 16 + 4 * g));
    }
    // rows of the values: tokens 16 tau + i, the workgroup's columns 32 j + 8 g and on (zeros past the last)
    __device__ Parts<NP> value_row(int base, int tau, int j) const {
        Parts<NP> o;
        if (p0 + 32 * j + 8 * g >= d.P) {
#pragma unroll
            for (int n = 0; n < NP; ++n) o.p[n] = b8v{};
        } else if constexpr (NP == 1) {
            o.p[0] = *reinterpret_cast<const b8v*>(sm + base + (tau * VJ + j) * 1024 + tile_slot(i, g) * 16);
        } else {
            const v4f* x = reinterpret_cast<const v4f*>(sm + base + ((16 * tau + i) * VS + 32 * j + 8 * g) * 4);
            o = __builtin_bit_cast(Parts<NP>, cut44<3>(x[0], x[1]));
        }
        return o;
    }
    __device__ static constexpr int terms(int na, int nb) {  // MFMAs of a product
        int n = 0;
        for (int s = 0; s < (na > nb ? na : nb); ++s)
            for (int k = 0; k < na; ++k) n += s - k >= 0 && s - k < nb;
        return n;
    }
    // Instructions do not move across; one MFMA, then VN others of the vector unit, N times.
    __device__ static void fence() { __builtin_amdgcn_sched_barrier(0); }
    template <int N, int VN>
    __device__ static void mix() {
#pragma unroll
        for (int m = 0; m < N; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, VN, 0);
        }
    }

    // ---------------------------------------------------------------- P
    // P's three tiles (tau, sigma) on and below the diagonal go round the waves, as D[s][t] (lane token
    // 16 tau + i), each into its half of an operand tile of row tau.  Powers come from registers: read
    // from a table, each waited for its own read (1500 cycles a chunk).
    __device__ void make_p() const {
        constexpr int MY = (3 + NW - 1) / NW;
#pragma unroll
        for (int m = 0; m < MY; ++m) {
            const int tile = w + NW * m, tau = tile > 0, sg = tile > 1;
            if (tile >= 3) break;
            Parts<NP> ko[2], qo[2];
            v4f x = zero4();
            ko[0] = row_op(oK, sg, 0);
            qo[0] = row_op(oQ, tau, 0);
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                if (j + 1 < KJ) {
                    ko[(j + 1) & 1] = row_op(oK, sg, j + 1);
                    qo[(j + 1) & 1] = row_op(oQ, tau, j + 1);
                }
                fence();
                x = mma(ko[j & 1], qo[j & 1], x);
                fence();
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                x[v] *= tau == sg ? near[v] : next[v];
            }
            const auto p = cut44<3>(x, x);
#pragma unroll
            for (int q = 0; q < 3; ++q)
                *reinterpret_cast<uint2*>(sm + oP + (q * TT + tau) * 1024 + lane * 16 + 8 * sg) =
                    *reinterpret_cast<const uint2*>(&p.p[q]);
        }
    }

    // ---------------------------------------------------------------- outputs
    // Outputs leave a chunk late and through LDS, where the waves' columns meet: whole rows, 16 bytes a
    // lane (16 columns a wave, in 32-byte pieces of sixteen rows, take three times as long to write).
    __device__ void keep_outputs(const v4f (&y)[NTILE][TT], int c) const {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int e = 0; e < NTILE; ++e) {
                // past the length zeros as they are: as products they would be NaN beside a NaN or an infinity
                const v4f z = whole(c) || c * C + 16 * t + i < len ? y[e][t] : zero4();
                Out* at = reinterpret_cast<Out*>(sm + oY + (16 * t + i) * YS) + wc + col_of(4 * g, e);
                io<typename std::conditional<sizeof(Out) == 2, BF16, F32>::type>::st4(at, 0, z);
            }
    }
    // f(place of a chunk, its row in dst)
    static constexpr int OV = PC * sizeof(Out) / 16, OROWS = THREADS / OV;  // vectors of a row, rows at a time
    __device__ void send_outputs(int c, bool zeros) const {
        const int r = threadIdx.x / OV, v = threadIdx.x % OV;
        if (p0 + v * (16 / static_cast<int>(sizeof(Out))) >= d.P) return;
        Out* const dst = static_cast<Out*>(a.dst) + b * a.os[0] + h * a.os[2] + p0;
        auto row = [&](int m) {
            return zeros ? make_uint4(0, 0, 0, 0)
                         : *reinterpret_cast<const uint4*>(sm + oY + (m * OROWS + r) * YS + v * 16);
        };
        if (whole(c)) {
            char* const base = reinterpret_cast<char*>(dst + first_row(c) * a.os[1]);
            const uint32_t step = a.os[1] * sizeof(Out), off = own_row(r, OROWS) * step + v * 16;
            uint4 x[C / OROWS];
#pragma unroll
            for (int m = 0; m < C / OROWS; ++m) x[m] = row(m);
#pragma unroll
            for (int m = 0; m < C / OROWS; ++m)
                *reinterpret_cast<uint4*>(base + shared_row(c, m * OROWS, OROWS) * step + off) = x[m];
        } else {
#pragma unroll
            for (int m = 0; m < C / OROWS; ++m) {
                const int u = c * C + m * OROWS + r;
                if (u < d.S)
                    *reinterpret_cast<uint4*>(reinterpret_cast<char*>(dst + (u < len ? token(u) : u) * a.os[1]) + v * 16) = row(m);
            }
        }
    }
    // ---------------------------------------------------------------- the derivative along the decay
    // <dy, dY> of a chunk without its outputs.  Of the pairs of tokens: sum (t-s) a^(t-s) (q_t.k_s) (dy_t.v_s), the
    // tiles round the waves like P's.  (Tokens past the n-th left out: zero times what may be no number any more in a
    // state that grows.)
    __device__ float pair_dots(int n) const {
        float sum = 0.0f;
        constexpr int MY = (3 + NW - 1) / NW;
#pragma unroll
        for (int m = 0; m < MY; ++m) {
            const int tile = w + NW * m, tau = tile > 0, sg = tile > 1;
            if (tile >= 3) break;
            v4f x = zero4(), z = zero4();
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                x = mma(row_op(oK, sg, j), row_op(oQ, tau, j), x);
                fence();  // (all of them at once would spill)
            }
#pragma unroll
            for (int j = 0; j < VJ; ++j) {
                z = mma(value_row(oV, sg, j), value_row(oP, tau, j), z);
                fence();
            }
            float pairs = 0.0f;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float by = (tau == sg ? near[v] : next[v]) * static_cast<float>(16 * (tau - sg) + i - 4 * g - v);
                pairs += by * x[v] * z[v];
            }
            sum += 16 * tau + i < n ? pairs : 0.0f;
        }
        return sum;
    }
    // Of the entry state: <T, W> + <H, W'> with W = sum a^(t+1) dy_t q_t^T and W' the same (t+1) times, whose tiles lie
    // as the state's: neither it nor T is cut into parts for it.  (By outputs Q T^T and Q H^T instead: 96 heads of
    // 2048 tokens, p = 64, r = 128, bf16 299 -> 243 us, fp32 554 -> 535.)
    __device__ float state_dots(const State& s, const State& ts) const {
        constexpr int G = GT, STEPS = RT / G;
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < NTILE; ++e) {
            v4f val[2];
            values(val, e, oP);
            const Parts<3> zo = weighted(val, qw), zt = weighted(val, qwt);
            Parts<NP> op[2][G];
#pragma unroll
            for (int m = 0; m < G; ++m) op[0][m] = col_op(m, oQ);
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                if (k + 1 < STEPS) {
#pragma unroll
                    for (int m = 0; m < G; ++m) op[(k + 1) & 1][m] = col_op((k + 1) * G + m, oQ);
                }
                v4f x[G], xt[G];
#pragma unroll
                for (int m = 0; m < G; ++m) x[m] = xt[m] = zero4();
                fence();
                mma_a(x, op[k & 1], zo);
                mma_a(xt, op[k & 1], zt);
                fence();
#pragma unroll
                for (int m = 0; m < G; ++m) {
                    const v4f y = ts[e][k * G + m] * x[m] + s[e][k * G + m] * xt[m];
                    sum += (y[0] + y[1]) + (y[2] + y[3]);
                }
            }
        }
        return sum;
    }

    // ---------------------------------------------------------------- the chunks
    __device__ void run() {
        // a segment after which the row ends (or that starts past its end) need not be carried
        if (!OUT && c1 == chunks) return;
        State s, ts[1];  // (ts: of the tangent)
        // entry states of the segments: [bh, seg], natural order (of the tangent: the states, then it)
        float* carry = a.carry ? a.carry + (bh * d.segs + seg) * a.cstep : nullptr;
        Ahead x;
        if (c0 < c1) fetch(x, c0);
        if constexpr (OUT) {
            if (d.segs > 1) {
                load_state(s, carry, a.csc, a.csr);
                if constexpr (TAN) load_state(ts[0], carry + size, a.csc, a.csr);
            } else {
                load_state(s, a.init ? a.init + bh * size : nullptr, a.csc, a.csr);
                if constexpr (TAN) load_state(ts[0], nullptr, 1, 1);
            }
        } else {
            load_state(s, nullptr, 1, 1);
            if constexpr (TAN) load_state(ts[0], nullptr, 1, 1);
        }
        float qf[TT];  // what a query's product with the state is scaled by
#pragma unroll
        for (int t = 0; t < TT; ++t) qf[t] = a.out * power(l2, 16 * t + i + 1 - a.rev);
        if constexpr (OUT) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int gap = i - 4 * g - v;
                near[v] = gap >= 0 ? a.out * a.in * power(l2, gap) : 0.0f;
                next[v] = a.out * a.in * power(l2, 16 + gap);
            }
            if (MODE == kTangent && threadIdx.x < C) {
                const int n = static_cast<int>(threadIdx.x) + 1;
                const float f = a.out * power(l2, n);
                qw[threadIdx.x] = f;
                qwt[threadIdx.x] = static_cast<float>(n) * f;
            }
            if (PLAIN && w == 0) {  // above P's diagonal
#pragma unroll
                for (int n = 0; n < 3; ++n)
                    *reinterpret_cast<uint2*>(sm + oP + n * TT * 1024 + lane * 16 + 8) = make_uint2(0, 0);
            }
        }
        put_factors(C);
        double kept = exp2(l2 * C);  // what the state keeps over a chunk, to more than 24 bits: it is raised
        float keep = static_cast<float>(kept), keep_lo = static_cast<float>(kept - keep);  // to the number of chunks
        double dot = 0.0;
#pragma unroll 1  // (a first chunk of its own, which the compiler makes otherwise, doubles the code: bf16 prompt 182 -> 185 us)
        for (int c = c0; c < c1; ++c) {
            const int n = len - c * C < C ? len - c * C : C;  // tokens of the chunk
            if constexpr (PLAIN)
                if (c > c0) send_outputs(c - 1, false);
            put(x, n);
            if (n < C) {
                put_factors(n);
                if (MODE == kTangent && static_cast<int>(threadIdx.x) >= n && threadIdx.x < C) qw[threadIdx.x] = qwt[threadIdx.x] = 0.0f;
                kept = exp2(l2 * n);
                keep = static_cast<float>(kept);
                keep_lo = static_cast<float>(kept - keep);
            }
            wait_barrier<63>();
            if (c + 1 < c1) fetch(x, c + 1);
            v4f y[NTILE][TT];
            if constexpr (PLAIN) {
                make_p();
                if (active) read_state(y, s, qf);
                wait_barrier<63>();  // P is here
            }
            if constexpr (MODE == kTangent) {
                // LDS addresses are made anew in every chunk: kept, beside two states and the parts of fp32 they
                // spill, and a reload waits for all that is being fetched (96 heads of 2048 tokens, r = 128, 535
                // -> 502 us; bf16, which does not spill, 243 -> 253)
                if constexpr (NP > 1 && R == 128) asm volatile("" : "+v"(i), "+v"(g));
                dot += pair_dots(n);
                fence();
                if (active) dot += state_dots(s, ts[0]);
                fence();
            }
            if (active) {
                advance(y, s, ts[0], n, keep, keep_lo);
                if constexpr (PLAIN) keep_outputs(y, c);
            }
            mfma_settle();
            wait_barrier<63>();  // everything of this chunk is read
        }
        if constexpr (!OUT) {
            store_state(s, carry, R, 1);
            if constexpr (TAN) store_state(ts[0], carry + size, R, 1);
            return;
        }
        // the segment that holds the row's last chunk, or the first one of an empty row
        const bool end = c1 == chunks && (c0 < c1 || seg == 0);
        if constexpr (PLAIN) {
            if (c0 < c1) send_outputs(c1 - 1, false);
            if (end && a.fin) store_state(s, a.fin + bh * size, a.csc, a.csr);
            const int last = (seg + 1) * d.seg_chunks < d.N ? (seg + 1) * d.seg_chunks : d.N;
            for (int c = c1 > seg * d.seg_chunks ? c1 : seg * d.seg_chunks; c < last; ++c) send_outputs(c, true);  // past the row's length
        } else if constexpr (MODE == kTangent) {
            if (end && a.d_final && active) {  // <d_final, T>
                const float* df = a.d_final + bh * size;
                float sum = 0.0f;
                each_state([&](int e, int rho, int col, int row) {
                    const v4f o = *reinterpret_cast<const v4f*>(df + col * static_cast<int64_t>(R) + row), z = ts[0][e][rho];
                    sum += o[0] * z[0] + o[1] * z[1] + o[2] * z[2] + o[3] * z[3];
                });
                dot += sum;
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o);
            double* sh = reinterpret_cast<double*>(sm);
            if (lane == 0) sh[w] = dot;
            __syncthreads();
            if (threadIdx.x == 0) {  // [h, (b, seg, column block)]
                double sum = 0.0;
                for (int m = 0; m < NW; ++m) sum += sh[m];
                const int pbs = d.P <= PC ? 1 : d.P / PC;
                a.dots[(static_cast<int64_t>(h) * d.B + b) * d.segs * pbs + seg * pbs + p0 / PC] = sum;
            }
        }
    }

    // y = scaled Q H^T as D[p][t]: lane token 16 t + i, rows columns col_of(4 g + v, e).  The state's parts
    // for a step are made while the matrix cores are at the step before.
    __device__ void read_state(v4f (&y)[NTILE][TT], const State& s, const float (&qf)[TT]) const {
#pragma unroll
        for (int e = 0; e < NTILE; ++e)
#pragma unroll
            for (int t = 0; t < TT; ++t) y[e][t] = zero4();
        Parts<NP> op[2][TT];
        Parts<3> hp[2][NTILE];
        auto parts = [&](int j) {
#pragma unroll
            for (int e = 0; e < NTILE; ++e) hp[j & 1][e] = cut44<3>(s[e][2 * j], s[e][2 * j + 1]);
        };
#pragma unroll
        for (int t = 0; t < TT; ++t) op[0][t] = row_op(oQ, t, 0);
        parts(0);
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            if (j + 1 < KJ) {
#pragma unroll
                for (int t = 0; t < TT; ++t) op[(j + 1) & 1][t] = row_op(oQ, t, j + 1);
            }
            fence();
#pragma unroll
            for (int e = 0; e < NTILE; ++e) mma_b(y[e], hp[j & 1][e], op[j & 1]);
            if (j + 1 < KJ) {
                parts(j + 1);
                mix<TT * NTILE * terms(3, NP), 28 / (TT * terms(3, NP)) + 1>();
            }
            fence();
        }
#pragma unroll
        for (int e = 0; e < NTILE; ++e)
#pragma unroll
            for (int t = 0; t < TT; ++t) y[e][t] *= qf[t];
    }

    // y <- y + P V, and the state over the chunk's n tokens.
    __device__ void advance(v4f (&y)[NTILE][TT], State& s, State& ts, int n, float keep, float keep_lo) const {
        Parts<NP> vo[NTILE];  // the values as operands, and times their powers
        Parts<3> zo[NTILE], zt[TAN ? NTILE : 1];
        v4f val[NTILE][2];
#pragma unroll
        for (int e = 0; e < NTILE; ++e) {
            values(val[e], e);
            if constexpr (PLAIN) {
                if constexpr (NP == 1)
                    vo[e].p[0] = join8(value4(0, e), value4(1, e));
                else
                    vo[e] = __builtin_bit_cast(Parts<NP>, cut44<3>(val[e][0], val[e][1]));
            }
        }
        auto fade = [&](int rho) {  // what the state keeps
#pragma unroll
            for (int e = 0; e < NTILE; ++e) {
                if constexpr (TAN) {
                    const v4f z = ts[e][rho] + static_cast<float>(n) * s[e][rho];
                    ts[e][rho] = z * keep + z * keep_lo;
                }
                s[e][rho] = s[e][rho] * keep + s[e][rho] * keep_lo;
            }
        };
        auto operands = [&]() {
#pragma unroll
            for (int e = 0; e < NTILE; ++e) {
                zo[e] = weighted(val[e], kf);
                if constexpr (TAN) zt[e] = weighted(val[e], kft);
            }
        };
        if constexpr (PLAIN) {
            // the vector unit fades the state and makes its operands meanwhile
            Parts<3> p[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    p[t].p[q] = *reinterpret_cast<const b8v*>(sm + oP + (q * TT + t) * 1024 + lane * 16);
            fence();
#pragma unroll
            for (int e = 0; e < NTILE; ++e) mma_b(y[e], vo[e], p);
#pragma unroll
            for (int rho = 0; rho < RT; ++rho) fade(rho);
            operands();
            mix<TT * NTILE * terms(NP, 3), 12>();
            fence();
        } else {
#pragma unroll
            for (int rho = 0; rho < RT; ++rho) fade(rho);
            operands();
        }
        constexpr int G = GT, STEPS = RT / G;
        Parts<NP> op[2][G];
#pragma unroll
        for (int m = 0; m < G; ++m) op[0][m] = col_op(m);
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            if (k + 1 < STEPS) {
#pragma unroll
                for (int m = 0; m < G; ++m) op[(k + 1) & 1][m] = col_op((k + 1) * G + m);
            }
            fence();
#pragma unroll
            for (int e = 0; e < NTILE; ++e) {
                mma_a(*reinterpret_cast<v4f(*)[G]>(&s[e][k * G]), op[k & 1], zo[e]);
                if constexpr (TAN) mma_a(*reinterpret_cast<v4f(*)[G]>(&ts[e][k * G]), op[k & 1], zt[e]);
            }
            fence();
        }
    }
};

// Tiles of columns of a wave for `columns` of a state with `rows`: two where 128 columns share a workgroup's
// operands (the parts of fp32 rows of 128 do not fit twice on a CU: two workgroups of 64 columns).
__host__ __device__ constexpr int linear_tiles(bool bf16, int columns, int rows) {
    return columns == 128 && (bf16 || rows <= 64) ? 2 : 1;
}
template <class IO, int COLUMNS, int ROWS>
constexpr int kLinearTiles = linear_tiles(in_parts<IO>() == 1, COLUMNS, ROWS);

// f(P, R) as constants
template <class F>
hipError_t by_widths(int p, int r, F&& f) {
    auto by_r = [&](auto pp) {
        switch (r) {
            case 16: return f(pp, std::integral_constant<int, 16>{});
            case 32: return f(pp, std::integral_constant<int, 32>{});
            case 64: return f(pp, std::integral_constant<int, 64>{});
            case 128: return f(pp, std::integral_constant<int, 128>{});
            default: return hipErrorInvalidValue;
        }
    };
    switch (p) {
        case 16: return by_r(std::integral_constant<int, 16>{});
        case 32: return by_r(std::integral_constant<int, 32>{});
        case 64: return by_r(std::integral_constant<int, 64>{});
        case 128: return by_r(std::integral_constant<int, 128>{});
        default: return hipErrorInvalidValue;
    }
}

}  // namespace ssd
