// Linear attention with a constant decay per head: the scan over chunks.
//
// Per head, with the state H [p, r] and a = exp(log_decay):
//   H_t = a H_{t-1} + v_t k_t^T,   y_t = scale H_t q_t,   H_{-1} = init.
// Over a chunk of C tokens with entry state H (tokens t, s counted inside it):
//   Y  = scale (a^{t+1} Q H^T + P V),   P_ts = a^{t-s} q_t.k_s (s <= t),
//   H' = a^C H + (a^{C-1-s} V)^T K.
// The gradient is the same scan three times.  With G_t the gradient of H_t through later outputs
// and the final state, G_t = a G_{t+1} + scale dy_t q_t^T:
//   d_q_t = scale H_t^T dy_t   (queries dy, keys v, values k, forwards from init),
//   d_v_t = G_t k_t            (queries k, keys q, values dy, backwards from d_final),
//   d_k_t = G_t^T v_t          (queries v, keys dy, values q, backwards; the state transposed).
// Backwards a state enters undecayed, so the powers are one lower for queries and one higher for
// keys, and what is left at the first token is d_init.
// The gradient of the decay is the derivative of the forward scan along it: T = dH / d log a,
//   T' = a^C (T + C H) + ((C-1-s) a^{C-1-s} V)^T K,
//   dY = scale (a^{t+1} Q (T + (t+1) H)^T + sum_s (t-s) P_ts V_s),   d_log_decay = <dy, dY> + <d_final, T_end>:
// every pair of tokens weighs in with its own distance, and nothing of the size of the positions cancels.
//
// Tokens past a row's length are zeros in every operand; their memory is not read.
#include <type_traits>

#include "delta_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {

namespace {

// Below this a log decay counts as this: its powers but the zeroth are zero in fp32, and 0 * -inf
// does not come up.
constexpr double kMinLogDecay = -1.0e4;

template <class IO>
__host__ __device__ constexpr int lin_chunk() { return in_parts<IO>() == 1 ? 64 : 32; }

// The eight XCDs take workgroups in turn and each has its own L2: give each a consecutive run of
// the work, so that the columns and value heads that read the same keys meet in one.
__device__ __forceinline__ int64_t xcd_order(int64_t blk, int64_t n) {
    const int64_t x = blk % 8, q = n / 8, rem = n % 8;
    return x * q + (x < rem ? x : rem) + blk / 8;
}

// a^n for the base-2 logarithm of a, in fp64
__device__ __forceinline__ float power(double log2a, int n) { return exp2_of(log2a * n); }

enum LinMode { kOutputs, kCarry, kTangent, kTangentCarry };

}  // namespace

// One workgroup: 64 NT value columns (or all of fewer) of one head, through the chunks of a segment.
template <class IO, int R, int NTILE, int MODE>
__global__ __launch_bounds__(256, 2) void k_linear(LinearShape d, LinearJobs jobs) {
    using T = typename IO::T;
    constexpr int C = lin_chunk<IO>(), NP = in_parts<IO>(), TT = C / 16, TJ = C / 32;
    constexpr int RP = R < 32 ? 32 : R, KJ = RP / 32, RT = RP / 16;
    constexpr int PC = 64 * NTILE, VJ = PC / 32;
    constexpr bool OUT = MODE == kOutputs || MODE == kTangent, TAN = MODE == kTangent || MODE == kTangentCarry;
    constexpr int QT = TT * KJ;                    // operand tiles of q or k, a part
    constexpr int TRI = TT == 4 ? 6 : 2;           // operand tiles of P, a part
    constexpr int VS = PC + 4;                     // floats of a row of v (fp32 io)
    constexpr int QBYTES = NP * QT * 1024, VBYTES = NP == 1 ? TT * VJ * 1024 : C * VS * 4;
    constexpr int PBYTES = OUT ? 3 * TRI * 1024 : 0;
    constexpr int oK = 0, oQ = oK + QBYTES, oV = oQ + (OUT ? QBYTES : 0), oP = oV + VBYTES,
                  oF = oP + PBYTES, LDS = oF + 4 * (3 * C + 4);
    __shared__ __align__(16) char sm[LDS];
    float* kf = reinterpret_cast<float*>(sm + oF);  // what a token's key adds to the state is scaled by
    float* kft = kf + C;                            // the same of the tangent
    float* pw = kft + C;                            // pw[n] = a^n, n <= C

    const LinearJob& a = jobs.job[blockIdx.y];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int pbs = d.P <= PC ? 1 : d.P / PC;
    const int per = MODE == kCarry || MODE == kTangentCarry ? d.segs - 1 : d.segs;
    const int64_t blk = xcd_order(blockIdx.x, gridDim.x);
    const int p0 = static_cast<int>(blk % pbs) * PC;
    const int seg = static_cast<int>(blk / pbs % per);
    const int64_t bh = blk / pbs / per;
    const int h = static_cast<int>(bh % d.H), b = static_cast<int>(bh / d.H);
    const int len = d.len ? static_cast<int>(d.len[b]) : d.S;
    const int chunks = (len + C - 1) / C;
    const int c0 = seg * d.seg_chunks < chunks ? seg * d.seg_chunks : chunks;
    const int c1 = c0 + d.seg_chunks < chunks ? c0 + d.seg_chunks : chunks;
    // a segment after which the row ends (or that starts past its end) need not be carried
    if (!OUT && c1 == chunks) return;

    const double l2 = (d.log_decay[h] < kMinLogDecay ? kMinLogDecay : static_cast<double>(d.log_decay[h])) * kLog2e;
    const int wc = w * 16 * NTILE;                       // this wave's first column, in the workgroup
    const bool active = p0 + wc < d.P;
    // column of row / operand lane m of column tile e, from the wave's first
    auto col_of = [](int m, int e) { return NTILE == 1 ? m : 8 * (m >> 2) + 4 * e + (m & 3); };

    // ---------------------------------------------------------------- state
    // s[e][rho][v]: row r = 32 (rho / 2) + 8 g + 4 (rho % 2) + v, column col_of(i, e)
    v4f s[NTILE][RT], ts[TAN ? NTILE : 1][TAN ? RT : 1];
    auto row_of = [&](int rho) { return 32 * (rho >> 1) + 8 * g + 4 * (rho & 1); };
    auto each_state = [&](auto&& f) {  // f(e, rho, column, row)
#pragma unroll
        for (int e = 0; e < NTILE; ++e)
#pragma unroll
            for (int rho = 0; rho < RT; ++rho)
                if (R >= 32 || row_of(rho) < R) f(e, rho, p0 + wc + col_of(i, e), row_of(rho));
    };
    auto load_state = [&](v4f(&x)[NTILE][RT], const float* src, int64_t sc, int64_t sr) {
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
    };
    auto store_state = [&](const v4f(&x)[NTILE][RT], float* dst, int64_t sc, int64_t sr) {
        if (!dst || !active) return;
        if (sr == 1)
            each_state([&](int e, int rho, int col, int row) { *reinterpret_cast<v4f*>(dst + col * sc + row) = x[e][rho]; });
        else
            each_state([&](int e, int rho, int col, int row) {
#pragma unroll
                for (int v = 0; v < 4; ++v) dst[col * sc + (row + v) * sr] = x[e][rho][v];
            });
    };
    const int64_t size = static_cast<int64_t>(d.P) * R;
    // entry states of the segments: [bh, seg], natural order (of the tangent: the states, then it)
    float* carry = a.carry ? a.carry + (bh * d.segs + seg) * a.cstep : nullptr;
    if constexpr (OUT) {
        if (d.segs > 1) {
            load_state(s, carry, a.csc, a.csr);
            if constexpr (TAN) load_state(ts, carry + size, a.csc, a.csr);
        } else {
            load_state(s, a.init ? a.init + bh * size : nullptr, a.csc, a.csr);
            if constexpr (TAN) load_state(ts, nullptr, 1, 1);
        }
    } else {
        load_state(s, nullptr, 1, 1);
        if constexpr (TAN) load_state(ts, nullptr, 1, 1);
    }

    // ---------------------------------------------------------------- loads, a chunk ahead
    auto token = [&](int u) {  // of place u of the row
        u = u < len ? u : len - 1;
        return static_cast<int64_t>(a.rev ? len - 1 - u : u);
    };
    typedef T raw8 __attribute__((ext_vector_type(8)));
    constexpr int PER = (QT + 3) / 4, VPER = NP == 1 ? TT * VJ / 4 : C * PC / 4 / 256;
    typedef T raw4 __attribute__((ext_vector_type(4)));
    raw8 kr[PER], qr[OUT ? PER : 1];
    typename std::conditional<NP == 1, raw8, raw4>::type vr[VPER];
    const int is = i ^ (4 * g);  // the token whose values lie in this lane's slot of an operand tile
    const T* kp = static_cast<const T*>(a.k) + b * a.ks[0] + (h / a.kdiv) * a.ks[2] + (8 * g < R ? 8 * g : 0);
    const T* qp = static_cast<const T*>(a.q) + b * a.qs[0] + (h / a.qdiv) * a.qs[2] + (8 * g < R ? 8 * g : 0);
    const T* vp = static_cast<const T*>(a.v) + b * a.vs[0] + (h / a.vdiv) * a.vs[2] + p0;
    auto fetch = [&](int c) {
#pragma unroll
        for (int m = 0; m < PER; ++m) {
            const int tile = w + 4 * m, tau = tile / KJ, j = tile % KJ;
            if (QT % 4 == 0 || tile < QT) {
                const int64_t t = token(c * C + 16 * tau + is);
                kr[m] = *reinterpret_cast<const raw8*>(kp + t * a.ks[1] + 32 * j);
                if constexpr (OUT) qr[m] = *reinterpret_cast<const raw8*>(qp + t * a.qs[1] + 32 * j);
            }
        }
#pragma unroll
        for (int m = 0; m < VPER; ++m) {
            if constexpr (NP == 1) {
                const int tile = w + 4 * m, tau = tile / VJ, col = 32 * (tile % VJ) + 8 * g;
                vr[m] = *reinterpret_cast<const raw8*>(vp + token(c * C + 16 * tau + is) * a.vs[1] +
                                                       (p0 + col < d.P ? col : 0));
            } else {
                const int at = threadIdx.x + 256 * m, col = 4 * (at % (PC / 4));
                vr[m] = *reinterpret_cast<const raw4*>(vp + token(c * C + at / (PC / 4)) * a.vs[1] +
                                                       (p0 + col < d.P ? col : 0));
            }
        }
    };
    auto put = [&](int c) {
        const int n = len - c * C;  // tokens left
#pragma unroll
        for (int m = 0; m < PER; ++m) {
            const int tile = w + 4 * m, tau = tile / KJ;
            if (QT % 4 == 0 || tile < QT) {
                const bool on = 16 * tau + is < n && (R >= 32 || 8 * g < R);
                const auto kx = parts_of<IO>(kr[m], on);
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    *reinterpret_cast<b8v*>(sm + oK + (q * QT + tile) * 1024 + lane * 16) = kx.p[q];
                if constexpr (OUT) {
                    const auto qx = parts_of<IO>(qr[m], on);
#pragma unroll
                    for (int q = 0; q < NP; ++q)
                        *reinterpret_cast<b8v*>(sm + oQ + (q * QT + tile) * 1024 + lane * 16) = qx.p[q];
                }
            }
        }
#pragma unroll
        for (int m = 0; m < VPER; ++m) {
            if constexpr (NP == 1) {
                const int tile = w + 4 * m, tau = tile / VJ;
                const auto vx = parts_of<IO>(vr[m], 16 * tau + is < n);
                *reinterpret_cast<b8v*>(sm + oV + tile * 1024 + lane * 16) = vx.p[0];
            } else {
                const int at = threadIdx.x + 256 * m, row = at / (PC / 4);
                v4f x = __builtin_bit_cast(v4f, vr[m]);
                if (row >= n) x = zero4();
                *reinterpret_cast<v4f*>(sm + oV + (row * VS + 4 * (at % (PC / 4))) * 4) = x;
            }
        }
    };
    // powers by which the tokens of a chunk of n reach its end
    auto put_factors = [&](int n) {
        if (threadIdx.x < C) {
            const int e = n - 1 - static_cast<int>(threadIdx.x);
            const float f = e >= 0 ? a.in * power(l2, e + a.rev) : 0.0f;
            kf[threadIdx.x] = f;
            if constexpr (TAN) kft[threadIdx.x] = static_cast<float>(e) * f;
        }
    };

    // ---------------------------------------------------------------- operands
    auto row_op = [&](int base, int tau, int j) {  // rows: tokens 16 tau + i
        Parts<NP> o;
#pragma unroll
        for (int n = 0; n < NP; ++n)
            o.p[n] = *reinterpret_cast<const b8v*>(sm + base + (n * QT + tau * KJ + j) * 1024 + tile_slot(i, g) * 16);
        return o;
    };
    auto col_op = [&](int rho, int j) {  // rows of state tile rho, k over the tokens of tiles 2 j and 2 j + 1
        Parts<NP> o;
        const int at = oK + (2 * j * KJ + (rho >> 1)) * 1024 + tile_slot(4 * g + (i >> 2), i & 3) * 16 + (rho & 1) * 8;
#pragma unroll
        for (int n = 0; n < NP; ++n)
            o.p[n] = join8(lds_col4(reinterpret_cast<const uint16_t*>(sm + at + n * QT * 1024)),
                           lds_col4(reinterpret_cast<const uint16_t*>(sm + at + (n * QT + KJ) * 1024)));
        return o;
    };
    // tokens 16 t + 4 g + v of column col_of(i, e), as they lie (bf16) or as values (fp32)
    auto value4 = [&](int t, int e) {
        if constexpr (NP == 1) {
            const int col = wc + (NTILE == 1 ? 4 * (i & 3) : 8 * (i & 3) + 4 * e);
            return lds_col4(reinterpret_cast<const uint16_t*>(
                sm + oV + (t * VJ + (col >> 5)) * 1024 + tile_slot(4 * g + (i >> 2), (col >> 3) & 3) * 16 +
                ((col >> 2) & 1) * 8));
        } else {
            const float* x = reinterpret_cast<const float*>(sm + oV) + (16 * t + 4 * g) * VS + wc + col_of(i, e);
            return v4f{x[0], x[VS], x[2 * VS], x[3 * VS]};
        }
    };

    // ---------------------------------------------------------------- the chunks
    float qf[TT];  // what a query's product with the state is scaled by
#pragma unroll
    for (int t = 0; t < TT; ++t) qf[t] = a.out * power(l2, 16 * t + i + 1 - a.rev);
    if (threadIdx.x <= C) pw[threadIdx.x] = a.out * a.in * power(l2, threadIdx.x);
    if constexpr (OUT) {  // halves of P's operand tiles above the diagonal
        constexpr int UP = TT / 2;
        if (threadIdx.x < 64 * UP) {
            const int tau = 2 * (threadIdx.x >> 6);
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                const int at = (n * TRI + tri_lower(tau, tau / 2)) * 1024 + lane * 16 + 8;
                *reinterpret_cast<uint2*>(sm + oP + at) = make_uint2(0, 0);
            }
        }
    }
    put_factors(C);
    double pass2 = exp2(l2 * C);  // what the state keeps over a chunk, to more than 24 bits: it is raised
    float keep = static_cast<float>(pass2), keep_lo = static_cast<float>(pass2 - keep);  // to the number of chunks
    double dot = 0.0;
    if (c0 < c1) fetch(c0);
    for (int c = c0; c < c1; ++c) {
        const int n = len - c * C < C ? len - c * C : C;  // tokens of the chunk
        put(c);
        if (n < C) {
            put_factors(n);
            pass2 = exp2(l2 * n);
            keep = static_cast<float>(pass2);
            keep_lo = static_cast<float>(pass2 - keep);
        }
        wait_barrier<63>();
        if (c + 1 < c1) fetch(c + 1);
        v4f y[NTILE][TT];
        if constexpr (OUT) {
            // P, 16 x 16 tiles (tau, sigma) on and below the diagonal in turn: D[s][t], lane token 16 tau + i
            constexpr int TILES = TT * (TT + 1) / 2;
#pragma unroll
            for (int m = 0; m < (TILES + 3) / 4; ++m) {
                const int tile = w + 4 * m;
                if (tile < TILES) {
                    const int tau = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0;
                    const int sg = tile - tau * (tau + 1) / 2;
                    v4f x = zero4();
#pragma unroll
                    for (int j = 0; j < KJ; ++j) x = mma(row_op(oK, sg, j), row_op(oQ, tau, j), x);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int gap = 16 * (tau - sg) + i - 4 * g - v;
                        x[v] = gap >= 0 ? x[v] * pw[gap >= 0 ? gap : 0] : 0.0f;
                        if constexpr (TAN) x[v] *= static_cast<float>(gap);
                    }
                    const int at = oP + tri_lower(tau, sg >> 1) * 1024 + lane * 16 + 8 * (sg & 1);
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        uint2 u;
                        u.x = f32x2_to_bf16x2(x[0], x[1]);
                        u.y = f32x2_to_bf16x2(x[2], x[3]);
                        *reinterpret_cast<uint2*>(sm + at + q * TRI * 1024) = u;
                        x -= v4f{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                                 __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)};
                    }
                }
            }
            // y = Q H^T as D[p][t]: lane token 16 tau + i, rows columns col_of(4 g + v, e)
#pragma unroll
            for (int e = 0; e < NTILE; ++e)
#pragma unroll
                for (int t = 0; t < TT; ++t) y[e][t] = zero4();
            if (active) {
                v4f yt[TAN ? NTILE : 1][TT];
                if constexpr (TAN) {
#pragma unroll
                    for (int t = 0; t < TT; ++t) yt[0][t] = zero4();
                }
                Parts<NP> op[2][TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) op[0][t] = row_op(oQ, t, 0);
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    if (j + 1 < KJ) {
#pragma unroll
                        for (int t = 0; t < TT; ++t) op[(j + 1) & 1][t] = row_op(oQ, t, j + 1);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int e = 0; e < NTILE; ++e) {
                        mma_b(y[e], split44<3>(s[e][2 * j], s[e][2 * j + 1]), op[j & 1]);
                        if constexpr (TAN) mma_b(yt[e], split44<3>(ts[e][2 * j], ts[e][2 * j + 1]), op[j & 1]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int e = 0; e < NTILE; ++e)
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        if constexpr (TAN) y[e][t] = yt[e][t] + static_cast<float>(16 * t + i + 1 - a.rev) * y[e][t];
                        y[e][t] *= qf[t];
                    }
            }
        }
        wait_barrier<63>();  // P is here
        if (active) {
            // the values as operands, and times their powers
            Parts<NP> vo[NTILE][TJ];
            Parts<3> zo[NTILE][TJ], zt[TAN ? NTILE : 1][TJ];
#pragma unroll
            for (int e = 0; e < NTILE; ++e)
#pragma unroll
                for (int j = 0; j < TJ; ++j) {
                    v4f x[2], z[2];
                    if constexpr (NP == 1) {
                        const s4 lo = value4(2 * j, e), hi = value4(2 * j + 1, e);
                        vo[e][j].p[0] = join8(lo, hi);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            x[0][v] = bf16_to_f32(lo[v]);
                            x[1][v] = bf16_to_f32(hi[v]);
                        }
                    } else {
                        x[0] = value4(2 * j, e);
                        x[1] = value4(2 * j + 1, e);
                        vo[e][j] = __builtin_bit_cast(Parts<NP>, split44<3>(x[0], x[1]));
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m) z[m] = x[m] * *reinterpret_cast<const v4f*>(kf + 16 * (2 * j + m) + 4 * g);
                    zo[e][j] = split44<3>(z[0], z[1]);
                    if constexpr (TAN) {
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            z[m] = x[m] * *reinterpret_cast<const v4f*>(kft + 16 * (2 * j + m) + 4 * g);
                        zt[e][j] = split44<3>(z[0], z[1]);
                    }
                }
            if constexpr (OUT) {
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int j = 0; j <= t / 2; ++j) {
                        Parts<3> p;
#pragma unroll
                        for (int q = 0; q < 3; ++q)
                            p.p[q] = *reinterpret_cast<const b8v*>(sm + oP +
                                                                   (q * TRI + tri_lower(t, j)) * 1024 + lane * 16);
#pragma unroll
                        for (int e = 0; e < NTILE; ++e) y[e][t] = mma(vo[e][j], p, y[e][t]);
                    }
            }
#pragma unroll
            for (int e = 0; e < NTILE; ++e)
#pragma unroll
                for (int rho = 0; rho < RT; ++rho) {
                    if constexpr (TAN) {
                        const v4f x = ts[e][rho] + static_cast<float>(n) * s[e][rho];
                        ts[e][rho] = x * keep + x * keep_lo;
                    }
                    s[e][rho] = s[e][rho] * keep + s[e][rho] * keep_lo;
                }
            constexpr int G = 2, STEPS = TJ * RT / G;  // state tiles at a time
            Parts<NP> op[2][G];
#pragma unroll
            for (int m = 0; m < G; ++m) op[0][m] = col_op(m, 0);
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                if (k + 1 < STEPS) {
#pragma unroll
                    for (int m = 0; m < G; ++m) op[(k + 1) & 1][m] = col_op((k + 1) % (RT / G) * G + m, (k + 1) / (RT / G));
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = 0; e < NTILE; ++e) {
                    mma_a(*reinterpret_cast<v4f(*)[G]>(&s[e][k % (RT / G) * G]), op[k & 1], zo[e][k / (RT / G)]);
                    if constexpr (TAN)
                        mma_a(*reinterpret_cast<v4f(*)[G]>(&ts[e][k % (RT / G) * G]), op[k & 1], zt[e][k / (RT / G)]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (OUT) {
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const int u = c * C + 16 * t + i;
                    if (u < d.S) {
                        const int64_t tok = u < len ? token(u) : u;
                        const int64_t at = b * a.os[0] + tok * a.os[1] + h * a.os[2] + p0 + wc;
                        float sum = 0.0f;
#pragma unroll
                        for (int e = 0; e < NTILE; ++e) {
                            // past the length zeros as they are: as products they would be NaN beside
                            // a NaN or an infinity
                            const v4f z = u < len ? y[e][t] : zero4();
                            const int64_t to = at + col_of(4 * g, e);
                            if constexpr (TAN) {
                                if (u < len) {
                                    const v4f o = io<IO>::ld4(static_cast<const T*>(a.dst), to);
                                    sum += o[0] * z[0] + o[1] * z[1] + o[2] * z[2] + o[3] * z[3];
                                }
                            } else if (a.wide) {
                                io<F32>::st4(static_cast<float*>(a.dst), to, z);
                            } else {
                                io<IO>::st4(static_cast<T*>(a.dst), to, z);
                            }
                        }
                        if constexpr (TAN) dot += sum;
                    }
                }
            }
        }
        mfma_settle();
        wait_barrier<63>();  // everything of this chunk is read
    }
    if constexpr (!OUT) {
        store_state(s, carry, R, 1);
        if constexpr (TAN) store_state(ts, carry + size, R, 1);
        return;
    }
    // the segment that holds the row's last chunk, or the first one of an empty row
    const bool end = c1 == chunks && (c0 < c1 || seg == 0);
    if constexpr (MODE == kOutputs) {
        if (end && a.fin) store_state(s, a.fin + bh * size, a.csc, a.csr);
        const int last = (seg + 1) * d.seg_chunks < d.N ? (seg + 1) * d.seg_chunks : d.N;
        int c = c1 > seg * d.seg_chunks ? c1 : seg * d.seg_chunks;
        if (active)
            for (; c < last; ++c) {  // chunks past the row's length
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const int u = c * C + 16 * t + i;
                    if (u < d.S) {
#pragma unroll
                        for (int e = 0; e < NTILE; ++e) {
                            const int64_t to = b * a.os[0] + u * a.os[1] + h * a.os[2] + p0 + wc + col_of(4 * g, e);
                            if (a.wide)
                                io<F32>::st4(static_cast<float*>(a.dst), to, zero4());
                            else
                                io<IO>::st4(static_cast<T*>(a.dst), to, zero4());
                        }
                    }
                }
            }
    } else {
        if (end && a.d_final && active) {  // <d_final, T>
            float sum = 0.0f;
            const float* df = a.d_final + bh * size;
#pragma unroll
            for (int e = 0; e < NTILE; ++e)
#pragma unroll
                for (int rho = 0; rho < RT; ++rho)
                    if (row_of(rho) < R) {
                        const v4f o = *reinterpret_cast<const v4f*>(df + (p0 + wc + col_of(i, e)) * static_cast<int64_t>(R) +
                                                                    row_of(rho));
                        sum += o[0] * ts[e][rho][0] + o[1] * ts[e][rho][1] + o[2] * ts[e][rho][2] + o[3] * ts[e][rho][3];
                    }
            dot += sum;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o);
        double* sh = reinterpret_cast<double*>(sm);
        if (lane == 0) sh[w] = dot;
        __syncthreads();
        // [h, (b, seg, column block)]
        if (threadIdx.x == 0)
            a.dots[(static_cast<int64_t>(h) * d.B + b) * d.segs * pbs + seg * pbs + p0 / PC] = sh[0] + sh[1] + sh[2] + sh[3];
    }
}

// From what each segment adds to a state to the states that the segments start from, in place.
// Layout [bh, seg, (H or H and T), p r]; a thread has four elements.
template <bool TAN>
__global__ __launch_bounds__(256) void k_linear_join(LinearShape d, LinearJobs jobs, int chunk) {
    const LinearJob& a = jobs.job[blockIdx.y];
    const int64_t size = static_cast<int64_t>(d.P) * d.R, quads = size / 4;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t bh = at / quads, q = at % quads;
    if (bh >= static_cast<int64_t>(d.B) * d.H) return;
    const int h = static_cast<int>(bh % d.H), b = static_cast<int>(bh / d.H);
    const int len = d.len ? static_cast<int>(d.len[b]) : d.S;
    const double l2 = (d.log_decay[h] < kMinLogDecay ? kMinLogDecay : static_cast<double>(d.log_decay[h])) * kLog2e;
    const int64_t tokens = static_cast<int64_t>(d.seg_chunks) * chunk;
    double x[4], t[4];
    const v4f x0 = a.init ? *reinterpret_cast<const v4f*>(a.init + bh * size + 4 * q) : zero4();
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        x[v] = x0[v];
        t[v] = 0.0;
    }
    const double f = exp2(l2 * tokens);
    for (int seg = 0; seg < d.segs; ++seg) {
        float* slot = a.carry + (bh * d.segs + seg) * a.cstep + 4 * q;
        const bool whole = (seg + 1) * tokens < len;  // only such a segment was carried, and is followed by another
        const v4f add = whole ? *reinterpret_cast<const v4f*>(slot) : zero4();
        *reinterpret_cast<v4f*>(slot) = v4f{static_cast<float>(x[0]), static_cast<float>(x[1]), static_cast<float>(x[2]),
                                            static_cast<float>(x[3])};
        if constexpr (TAN) {
            const v4f tadd = whole ? *reinterpret_cast<const v4f*>(slot + size) : zero4();
            *reinterpret_cast<v4f*>(slot + size) = v4f{static_cast<float>(t[0]), static_cast<float>(t[1]),
                                                       static_cast<float>(t[2]), static_cast<float>(t[3])};
#pragma unroll
            for (int v = 0; v < 4; ++v) t[v] = f * (t[v] + static_cast<double>(tokens) * x[v]) + tadd[v];
        }
        if (!whole) return;
#pragma unroll
        for (int v = 0; v < 4; ++v) x[v] = f * x[v] + add[v];
    }
}

// d_decay[h] from the workgroups' sums, one after the other.
__global__ __launch_bounds__(64) void k_linear_decay(const double* dots, int per, float* d_decay) {
    double x = 0.0;
    for (int n = threadIdx.x; n < per; n += 64) x += dots[static_cast<int64_t>(blockIdx.x) * per + n];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
    if (threadIdx.x == 0) d_decay[blockIdx.x] = static_cast<float>(x);
}

// Gradients of shared key heads: [tokens, hk, grp, r] fp32 summed over grp.
template <class IO>
__global__ __launch_bounds__(256) void k_linear_share(const float* src, int64_t rows, int grp, int r,
                                                      typename IO::T* dst) {
    const int quads = r / 4;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < rows * quads;
         at += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = at / quads;
        const int q = static_cast<int>(at % quads);
        v4f x = zero4();
        for (int m = 0; m < grp; ++m) x += *reinterpret_cast<const v4f*>(src + (row * grp + m) * r + 4 * q);
        io<IO>::st4(dst, row * r + 4 * q, x);
    }
}

namespace {

template <class IO, int R, int MODE>
hipError_t run_r(const LinearShape& d, const LinearJobs& jobs, hipStream_t st) {
    const int per = MODE == kCarry || MODE == kTangentCarry ? d.segs - 1 : d.segs;
    const int64_t heads = static_cast<int64_t>(d.B) * d.H * per;
    if constexpr (MODE == kOutputs || MODE == kCarry) {
        if (d.P == 128) {
            k_linear<IO, R, 2, MODE><<<dim3(static_cast<unsigned>(heads), jobs.n), 256, 0, st>>>(d, jobs);
            return hipGetLastError();
        }
    }
    const int pbs = d.P <= 64 ? 1 : d.P / 64;
    k_linear<IO, R, 1, MODE><<<dim3(static_cast<unsigned>(heads * pbs), jobs.n), 256, 0, st>>>(d, jobs);
    return hipGetLastError();
}

template <int MODE>
hipError_t run(const LinearShape& d, const LinearJobs& jobs, hipStream_t st) {
    auto by_io = [&](auto r) {
        constexpr int R = decltype(r)::value;
        return d.io == 1 ? run_r<BF16, R, MODE>(d, jobs, st) : run_r<F32, R, MODE>(d, jobs, st);
    };
    switch (d.R) {
        case 16: return by_io(std::integral_constant<int, 16>{});
        case 32: return by_io(std::integral_constant<int, 32>{});
        case 64: return by_io(std::integral_constant<int, 64>{});
        case 128: return by_io(std::integral_constant<int, 128>{});
        default: return hipErrorInvalidValue;
    }
}

int chunk_of(int io) { return io == 1 ? lin_chunk<BF16>() : lin_chunk<F32>(); }

}  // namespace

int linear_chunk(int io) { return chunk_of(io); }

int linear_segments(const LinearShape& d, int jobs) {
    const int64_t wgs = static_cast<int64_t>(d.B) * d.H * jobs;
    if (d.N < 16 || wgs > 256) return 1;
    int64_t n = 512 / wgs;
    if (n > d.N / 8) n = d.N / 8;
    return n < 2 ? 1 : static_cast<int>(n);
}

hipError_t launch_linear_scan(const LinearShape& d, const LinearJobs& jobs, hipStream_t st) {
    return run<kOutputs>(d, jobs, st);
}
hipError_t launch_linear_carry(const LinearShape& d, const LinearJobs& jobs, bool tangent, hipStream_t st) {
    return tangent ? run<kTangentCarry>(d, jobs, st) : run<kCarry>(d, jobs, st);
}
hipError_t launch_linear_tangent(const LinearShape& d, const LinearJobs& jobs, hipStream_t st) {
    return run<kTangent>(d, jobs, st);
}
hipError_t launch_linear_join(const LinearShape& d, const LinearJobs& jobs, bool tangent, hipStream_t st) {
    const int64_t quads = static_cast<int64_t>(d.B) * d.H * d.P * d.R / 4;
    const dim3 grid(static_cast<unsigned>((quads + 255) / 256), jobs.n);
    if (tangent)
        k_linear_join<true><<<grid, 256, 0, st>>>(d, jobs, chunk_of(d.io));
    else
        k_linear_join<false><<<grid, 256, 0, st>>>(d, jobs, chunk_of(d.io));
    return hipGetLastError();
}
int linear_dots(const LinearShape& d) { return d.B * d.segs * (d.P <= 64 ? 1 : d.P / 64); }
hipError_t launch_linear_decay(const LinearShape& d, const double* dots, float* d_decay, hipStream_t st) {
    k_linear_decay<<<dim3(d.H), 64, 0, st>>>(dots, linear_dots(d), d_decay);
    return hipGetLastError();
}
hipError_t launch_linear_share(const LinearShape& d, int kheads, int r, const float* src, void* dst, hipStream_t st) {
    const int64_t rows = static_cast<int64_t>(d.B) * d.S * kheads, items = rows * (r / 4);
    const dim3 grid(static_cast<unsigned>(items / 256 + 1 < 8192 ? items / 256 + 1 : 8192));
    if (d.io == 1)
        k_linear_share<BF16><<<grid, 256, 0, st>>>(src, rows, d.H / kheads, r, static_cast<uint16_t*>(dst));
    else
        k_linear_share<F32><<<grid, 256, 0, st>>>(src, rows, d.H / kheads, r, static_cast<float*>(dst));
    return hipGetLastError();
}

}  // namespace ssd
