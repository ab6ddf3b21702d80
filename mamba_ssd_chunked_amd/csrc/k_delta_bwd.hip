// The gated delta rule: gradients of one chunk from its entry state H, the gradient dH of the
// state that leaves it, E and dZ (all from the two recurrences of the backward).
//
// With U = beta E, dR = beta dZ (= dV) and the decay D_ts = exp(G_t - G_s):
//   dP = dY U^T (s <= t),  dAb = -dR U^T (s < t),  dS = scale D dP,  dKK = D dAb,
//   dQ  = scale e^G dY H + dS K,
//   dK  = (-e^G dR H + dKK K) + (e^{G_L - G} U dH + dS^T Q + dKK^T K),
//   dbeta_t = dZ_t . E_t,
//   dG_t = q_t . (scale e^G dY H)_t + k_t . (-e^G dR H)_t + sum_s W_ts - sum_s W_st - w_t,
//          W = dP P + dAb Ab off the diagonal, w_t = k_t . (e^{G_L - G} U dH)_t,
//   dG_L += sum_t w_t + e^{G_L} <dH, H>,  and d_g is the suffix sum of dG in the chunk:
//   d_g_t = sum_{s >= t} (dG_s + w_s) + sum_{s < t} w_s + e^{G_L} <dH, H>
// where the w of later tokens, which would cancel, never appear.
//
// One workgroup of eight waves per (b, key head, chunk); the value heads that share the key
// head are added up in its registers, in order.  It moves 2.7 GB in 655 us, 4.1 TB/s (bf16, 160
// heads of 64 chunks, p = 64, r = 128; fp32, 96 heads of 32 chunks: 310 us), bound by HBM and by
// cutting H, dH, E and dZ into parts.  Value columns go through LDS 32 at a time; a
// wave owns one 16-row tile of r and its tiles of tokens, so H and dH are read once, straight
// into operand registers.
#include <type_traits>

#include "delta_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {

namespace {

constexpr int PB = 32;       // value columns staged at a time
constexpr int GW = 8;        // waves of a workgroup
constexpr int LP = PB + 8;   // their LDS row stride
constexpr int LS = DL + 8;   // row stride of a 64 x 64 part

template <int N>
__device__ __forceinline__ void store_parts4(uint16_t* dst, int part_stride, v4f x) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint2 w;
        w.x = f32x2_to_bf16x2(x[0], x[1]);
        w.y = f32x2_to_bf16x2(x[2], x[3]);
        *reinterpret_cast<uint2*>(dst + n * part_stride) = w;
        if (n + 1 < N)
            x -= v4f{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
    }
}
template <int N>
__device__ __forceinline__ v4f sum_parts4(const uint16_t* src, int part_stride) {
    v4f x = zero4();
#pragma unroll
    for (int n = N - 1; n >= 0; --n) x += io<BF16>::ld4(src + n * part_stride, 0);
    return x;
}

// Operand rows 16 tile + i, k = k0 + 8 g .., of a row-major LDS matrix of parts.
template <int N>
__device__ __forceinline__ Parts<N> rows8(const uint16_t* m, int part_stride, int ld, int row, int col) {
    Parts<N> o;
#pragma unroll
    for (int n = 0; n < N; ++n) o.p[n] = *reinterpret_cast<const b8v*>(m + n * part_stride + row * ld + col);
    return o;
}
// Operand rows = columns col0 + i, k = rows row0 + 8 g ..: the transposed matrix.
template <int N>
__device__ __forceinline__ Parts<N> cols8(const uint16_t* m, int part_stride, int ld, int row0, int col0, int i, int g) {
    Parts<N> o;
    const uint16_t* at = m + (row0 + 8 * g + (i >> 2)) * ld + col0 + 4 * (i & 3);
#pragma unroll
    for (int n = 0; n < N; ++n) o.p[n] = join8(lds_col4(at + n * part_stride), lds_col4(at + n * part_stride + 4 * ld));
    return o;
}

}  // namespace

// bf16 without shared heads: 76 KB of LDS and, held to 128 registers, two workgroups on a CU (655 us
// for 160 heads of 64 chunks with p = 64, r = 128, against 999 us for one of four waves; sixteen
// waves on one chunk: 909 us).  fp32 takes 152 KB of LDS: one workgroup a CU.
template <class IO, int R, bool SHARED>
__global__ __launch_bounds__(GW * 64, in_parts<IO>() == 1 && !SHARED ? 4 : 2) void k_delta_grad(
    DeltaShape d, DeltaScan<typename IO::T> a, typename IO::T* __restrict__ d_q, typename IO::T* __restrict__ d_k,
    typename IO::T* __restrict__ d_v, float* __restrict__ d_g, float* __restrict__ d_beta) {
    using T = typename IO::T;
    constexpr int NP = in_parts<IO>(), RP = R < 32 ? 32 : R, KJ = RP / 32;
    constexpr int RT = R / 16, ITEMS = RT * 4 < GW ? 1 : RT * 4 / GW, V = RP / 8, NTHR = GW * 64;
    // Loading a block ahead takes the registers of a second workgroup on the CU, which hides the
    // loads better (160 heads of 64 chunks, bf16, p = 64, r = 128: 655 against 857 us), except where
    // a workgroup goes through several value heads (16 heads in 8, 777 tokens: 45 against 38 us).
    constexpr bool AHEAD = SHARED;
    constexpr int CT = PB / GW;  // value columns of one thread's piece of a token row
    constexpr int PAIRS = 2;     // pair tiles of one wave
    constexpr int KQ = 4 * KJ * DTILE, UP = DL * LP, SP = DL * LS;
    __shared__ __align__(16) uint16_t sK[NP * KQ], sQ[NP * KQ];
    __shared__ __align__(16) union {
        struct {
            uint16_t U[3 * UP], Z[3 * UP], Y[NP * UP];
        } v;
        uint16_t S[3 * SP];
    } sm;
    __shared__ float sCf[3 * DL + 1];  // e^G, e^{G_L - G}, beta, e^{G_L}
    __shared__ double sG[DL];
    __shared__ float sLoc[RT][DL], sWr[RT][DL], sRow[4][DL], sCol[4][DL], sDot[GW];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The lane's place, made anew in each phase from a value the compiler cannot see through: kept
    // over the phases, the addresses it derives from them would take every register.
    int tid, lane, i, g, vt, vp;
    auto here = [&]() {
        tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        lane = tid & 63;
        i = lane & 15;
        g = lane >> 4;
        vt = tid / GW;
        vp = CT * (tid % GW);
    };
    here();
    const unsigned blk = blockIdx.x, n_chunks = d.N, n_heads = d.HK;
    const int c = blk % n_chunks, hk = blk / n_chunks % n_heads, b = blk / n_chunks / n_heads;
    const int64_t t0 = static_cast<int64_t>(c) * DL, row0 = static_cast<int64_t>(b) * d.S + t0;
    const int grp = SHARED ? d.H / d.HK : 1;
    const int all = static_cast<int>(d.S - t0 < DL ? d.S - t0 : DL);  // rows of the tensors
    const int64_t left = (a.len ? a.len[b] : d.S) - t0;
    const int L = left < 0 ? 0 : (left > DL ? DL : static_cast<int>(left));
    if (L == 0) {  // past the row's length
        for (int x = tid; x < all * (R / 4); x += NTHR) {
            const int64_t at = ((row0 + x / (R / 4)) * d.HK + hk) * R + 4 * (x % (R / 4));
            io<IO>::st4(d_q, at, zero4());
            io<IO>::st4(d_k, at, zero4());
        }
        for (int hh = 0; hh < grp; ++hh) {
            const int h = hk * grp + hh;
            for (int x = tid; x < all * (d.P / 4); x += NTHR)
                io<IO>::st4(d_v, ((row0 + x / (d.P / 4)) * d.H + h) * d.P + 4 * (x % (d.P / 4)), zero4());
            if (tid < all) d_g[(row0 + tid) * d.H + h] = d_beta[(row0 + tid) * d.H + h] = 0.0f;
        }
        return;
    }
    const int rho = w * ITEMS / 4, tt0 = (w * ITEMS) & 3;  // this wave's r tile and first token tile
    const bool act = rho < RT;
    // the causal pair tiles (token tile tau, source tile sigma) of this wave: of ten, w and w + GW
    auto tau_of = [](int idx) { return idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3; };
    auto pairs = [&](auto f) {
#pragma unroll
        for (int m = 0; m < PAIRS; ++m) {
            const int idx = w + m * GW, tau = tau_of(idx);
            if (idx < 10) f(m, tau, idx - tau * (tau + 1) / 2);
        }
    };

    // one block of value columns: this thread's piece of the token rows, and its wave's rows of H and dH
    v4f e, z, y, h0, h1, g0, g1;
    auto fetch = [&](int hh, int p0) {
        const int h = hk * grp + hh;
        const int64_t ch = (static_cast<int64_t>(b) * d.H + h) * d.N + c;
        const int p = p0 + vp;
        e = z = y = h0 = h1 = g0 = g1 = zero4();
        if (p < d.P) {
            const int64_t at = (ch * DL + vt) * d.P + p, ay = ((row0 + vt) * d.H + h) * d.P + p;
            e = *reinterpret_cast<const v4f*>(a.E + at);
            z = *reinterpret_cast<const v4f*>(a.dZ + at);
            if (vt < L) y = io<IO>::ld4(a.dy, ay);
        }
        const int ph = p0 + 8 * g;
        if (act && ph < d.P) {
            const int64_t at = (ch * R + 16 * rho + i) * d.P + ph;
            h0 = *reinterpret_cast<const v4f*>(a.H + at);
            h1 = *reinterpret_cast<const v4f*>(a.H + at + 4);
            g0 = *reinterpret_cast<const v4f*>(a.dH + at);
            g1 = *reinterpret_cast<const v4f*>(a.dH + at + 4);
        }
    };
    {  // keys and queries in tiles of 16 tokens x 32, zeros past the length
        typedef T raw8 __attribute__((ext_vector_type(8)));
        constexpr int KV = (DL * V + NTHR - 1) / NTHR;
        raw8 kr[KV], qr[KV];
#pragma unroll
        for (int m = 0; m < KV; ++m) {
            const int t = (tid + m * NTHR) / V, col = 8 * (tid % V), row = t < L ? t : L - 1, from = col < R ? col : 0;
            kr[m] = *reinterpret_cast<const raw8*>(a.k + b * d.ks[0] + (t0 + row) * d.ks[1] + hk * d.ks[2] + from);
            qr[m] = *reinterpret_cast<const raw8*>(a.q + b * d.qs[0] + (t0 + row) * d.qs[1] + hk * d.qs[2] + from);
        }
        if (AHEAD) fetch(0, 0);
#pragma unroll
        for (int m = 0; m < KV; ++m) {
            const int t = (tid + m * NTHR) / V, col = 8 * (tid % V);
            if (t < DL) {
                const auto kp = parts_of<IO>(kr[m], t < L && col < R), qp = parts_of<IO>(qr[m], t < L && col < R);
                const int at = ((t >> 4) * KJ + (col >> 5)) * DTILE + tile_slot(t & 15, (col >> 3) & 3) * 8;
#pragma unroll
                for (int x = 0; x < NP; ++x) {
                    *reinterpret_cast<b8v*>(sK + x * KQ + at) = kp.p[x];
                    *reinterpret_cast<b8v*>(sQ + x * KQ + at) = qp.p[x];
                }
            }
        }
    }
    auto kq_rows = [&](const uint16_t* m, int tile, int j) {  // operand rows: tokens 16 tile + i
        Parts<NP> o;
#pragma unroll
        for (int x = 0; x < NP; ++x)
            o.p[x] = *reinterpret_cast<const b8v*>(m + x * KQ + (tile * KJ + j) * DTILE + tile_slot(i, g) * 8);
        return o;
    };
    auto kq_cols = [&](const uint16_t* m, int j) {  // rows: r = 16 rho + i, k over the tokens 32 j + 8 g ..
        Parts<NP> o;
        const int t = 32 * j + 8 * g + (i >> 2);
        const uint16_t* at = m + ((t >> 4) * KJ + (rho >> 1)) * DTILE + 4 * (i & 1);
        const int gg = 2 * (rho & 1) + ((i & 3) >> 1);
#pragma unroll
        for (int x = 0; x < NP; ++x)
            o.p[x] = join8(lds_col4(at + x * KQ + tile_slot(t & 15, gg) * 8),
                           lds_col4(at + x * KQ + tile_slot((t & 15) + 4, gg) * 8));
        return o;
    };
    v4f dq[SHARED ? ITEMS : 1], dk[SHARED ? ITEMS : 1];
#pragma unroll
    for (int m = 0; m < (SHARED ? ITEMS : 1); ++m) dq[m] = dk[m] = zero4();

    for (int hh = 0; hh < grp; ++hh) {
        const int h = hk * grp + hh;
        const int64_t ch = (static_cast<int64_t>(b) * d.H + h) * d.N + c;
        const float* cf = a.coef + ch * DCOEF;
        if (hh > 0) __syncthreads();
        if (tid <= 3 * DL) sCf[tid] = cf[tid];
        if (tid < DL) sG[tid] = reinterpret_cast<const double*>(cf + DCF)[tid];
        const float be = cf[2 * DL + vt];
        v4f aq[ITEMS], akr[ITEMS], akw[ITEMS], dP[PAIRS], dA[PAIRS];
#pragma unroll
        for (int m = 0; m < PAIRS; ++m) dP[m] = dA[m] = zero4();
#pragma unroll
        for (int m = 0; m < ITEMS; ++m) aq[m] = akr[m] = akw[m] = zero4();
        float db = 0.0f, hdh = 0.0f;
        for (int p0 = 0; p0 < d.P; p0 += PB) {
            here();
            if (!AHEAD) fetch(hh, p0);
            if (p0 > 0) __syncthreads();
            db += e[0] * z[0] + e[1] * z[1] + e[2] * z[2] + e[3] * z[3];
            e *= be;
            z *= be;
            if (p0 + vp < d.P && vt < all)  // past the length zeros as they are, beside NaN too
                io<IO>::st4(d_v, ((row0 + vt) * d.H + h) * d.P + p0 + vp, vt < L ? z : zero4());
            store_parts4<3>(sm.v.U + vt * LP + vp, UP, e);
            store_parts4<3>(sm.v.Z + vt * LP + vp, UP, z);
            store_parts4<NP>(sm.v.Y + vt * LP + vp, UP, y);
            if (tt0 == 0) {
#pragma unroll
                for (int v = 0; v < 4; ++v) hdh += h0[v] * g0[v] + h1[v] * g1[v];
            }
            const auto hp = split44<3>(h0, h1);
            const auto gp = split44<3>(g0, g1);
            if (AHEAD) {  // the next block's, under way while this one is multiplied
                if (p0 + PB < d.P)
                    fetch(hh, p0 + PB);
                else if (hh + 1 < grp)
                    fetch(hh + 1, 0);
            }
            __syncthreads();
            if (act) {
#pragma unroll
                for (int m = 0; m < ITEMS; ++m) {
                    const int row = 16 * (tt0 + m) + i;
                    aq[m] = mma(hp, rows8<NP>(sm.v.Y, UP, LP, row, 8 * g), aq[m]);
                    akr[m] = mma(hp, rows8<3>(sm.v.Z, UP, LP, row, 8 * g), akr[m]);
                    akw[m] = mma(gp, rows8<3>(sm.v.U, UP, LP, row, 8 * g), akw[m]);
                }
            }
            pairs([&](int m, int tau, int sig) {
                const auto u = rows8<3>(sm.v.U, UP, LP, 16 * sig + i, 8 * g);
                dP[m] = mma(u, rows8<NP>(sm.v.Y, UP, LP, 16 * tau + i, 8 * g), dP[m]);
                dA[m] = mma(u, rows8<3>(sm.v.Z, UP, LP, 16 * tau + i, 8 * g), dA[m]);
            });
            mfma_settle();
        }
        here();
        // results D[r][t] (lane token 16 tt + i, rows r = 16 rho + 4 g + v)
        if (act) {
#pragma unroll
            for (int m = 0; m < ITEMS; ++m) {
                const int t = 16 * (tt0 + m) + i;
                const int at = ((tt0 + m) * KJ + (rho >> 1)) * DTILE + tile_slot(i, 2 * (rho & 1) + (g >> 1)) * 8 +
                               4 * (g & 1);
                const float eg = sCf[t], tail = sCf[DL + t];
                aq[m] *= d.scale * eg;
                akr[m] *= -eg;
                akw[m] *= tail;
                const v4f q4 = sum_parts4<NP>(sQ + at, KQ), k4 = sum_parts4<NP>(sK + at, KQ);
                float loc = 0.0f, wr = 0.0f;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    loc += q4[v] * aq[m][v] + k4[v] * akr[m][v];
                    wr += k4[v] * akw[m][v];
                }
                loc = sum_over_g(loc);
                wr = sum_over_g(wr);
                if (g == 0) {
                    sLoc[rho][t] = loc;
                    sWr[rho][t] = wr;
                }
                akr[m] += akw[m];  // the inter-chunk part of d_k
            }
        }
        if (tt0 == 0) {
            hdh = sum_over_lanes<16>(hdh);
            hdh = sum_over_g(hdh);
        }
        if (lane == 0) sDot[w] = hdh;
        here();
        pairs([&](int m, int tau, int sig) {  // pair tile D[s][t] (lane token 16 tau + i, sources 16 sig + 4 g + v)
            v4f kk = zero4(), qk = zero4();
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                const auto ks = kq_rows(sK, sig, j);
                kk = mma(ks, kq_rows(sK, tau, j), kk);
                qk = mma(ks, kq_rows(sQ, tau, j), qk);
            }
            const int t = 16 * tau + i;
            float wrow = 0.0f;
            v4f wcol;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int s = 16 * sig + 4 * g + v;
                const float e2 = s <= t ? exp2_of(sG[t] - sG[s]) : 0.0f;
                const float es = s < t ? e2 : 0.0f;
                const float x = es * (d.scale * dP[m][v] * qk[v] - dA[m][v] * kk[v]);
                wrow += x;
                wcol[v] = sum_over_lanes<16>(x);
                dP[m][v] *= d.scale * e2;
                dA[m][v] *= -es;
            }
            wrow = sum_over_g(wrow);
            if (g == 0) sRow[sig][t] = wrow;
            if (i == 0) *reinterpret_cast<v4f*>(&sCol[tau][16 * sig + 4 * g]) = wcol;
        });
        db = sum_over_lanes<8>(db);  // the GW threads of a token row
        if (tid % GW == 0 && vt < all) d_beta[(row0 + vt) * d.H + h] = vt < L ? db : 0.0f;
#pragma unroll
        for (int which = 0; which < 2; ++which) {  // dS, then dKK
            here();
            __syncthreads();
            pairs([&](int m, int tau, int sig) {
                uint16_t* at = sm.S + (16 * tau + i) * LS + 16 * sig + 4 * g;
                store_parts4<3>(at, SP, which ? dA[m] : dP[m]);
                if (sig == tau && (tau & 1) == 0) store_parts4<3>(at + 16, SP, zero4());
            });
            __syncthreads();
            if (which == 0 && w == GW - 1) {
                float loc = 0.0f, wr = 0.0f, hd = 0.0f;
#pragma unroll
                for (int m = 0; m < RT; ++m) {
                    loc += sLoc[m][lane];
                    wr += sWr[m][lane];
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (m <= g) loc += sRow[m][lane];
                    if (m >= g) loc -= sCol[m][lane];
                }
#pragma unroll
                for (int m = 0; m < RT; ++m) hd += sDot[m * 4 / ITEMS];
                double suf = loc, pre = wr;
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) {
                    const double u = __shfl_down(suf, o), x = __shfl_up(pre, o);
                    if (lane + o < 64) suf += u;
                    if (lane >= o) pre += x;
                }
                pre = __shfl_up(pre, 1);
                if (lane == 0) pre = 0.0;
                double out = suf + pre + static_cast<double>(sCf[3 * DL]) * hd;
                // a decay of 0, which forgets the state: exactly zero, where the sums leave their rounding
                if (exp2_of(sG[lane] - (lane > 0 ? sG[lane - 1] : 0.0)) == 0.0f) out = 0.0;
                if (lane < all) d_g[(row0 + lane) * d.H + h] = lane < L ? static_cast<float>(out) : 0.0f;
            }
            if (act) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const auto kt = kq_cols(sK, j);
                    Parts<NP> xt;
                    if (which == 0) xt = kq_cols(sQ, j);
#pragma unroll
                    for (int m = 0; m < ITEMS; ++m) {
                        const int tt = tt0 + m;
                        if (j <= tt / 2) {
                            const auto x = rows8<3>(sm.S, SP, LS, 16 * tt + i, 32 * j + 8 * g);
                            if (which == 0) aq[m] = mma(kt, x, aq[m]);
                            else akr[m] = mma(kt, x, akr[m]);
                        }
                        if (j >= tt / 2) {
                            const auto x = cols8<3>(sm.S, SP, LS, 32 * j, 16 * tt, i, g);
                            akr[m] = mma(which == 0 ? xt : kt, x, akr[m]);
                        }
                    }
                }
            }
        }
        if (act) {
#pragma unroll
            for (int m = 0; m < ITEMS; ++m) {
                if constexpr (SHARED) {
                    dq[m] += aq[m];
                    dk[m] += akr[m];
                }
                const int t = 16 * (tt0 + m) + i;
                if (hh + 1 == grp && t < all) {
                    const int64_t at = ((row0 + t) * d.HK + hk) * R + 16 * rho + 4 * g;
                    io<IO>::st4(d_q, at, t >= L ? zero4() : SHARED ? dq[SHARED ? m : 0] : aq[m]);
                    io<IO>::st4(d_k, at, t >= L ? zero4() : SHARED ? dk[SHARED ? m : 0] : akr[m]);
                }
            }
        }
    }
}

namespace {

template <class IO>
hipError_t grad_io(const DeltaShape& d, const DeltaBufs& f, hipStream_t st) {
    using T = typename IO::T;
    DeltaScan<T> a{};
    a.q = static_cast<const T*>(f.q);
    a.k = static_cast<const T*>(f.k);
    a.dy = static_cast<const T*>(f.dy);
    a.len = f.len;
    a.coef = f.coef;
    a.H = f.H;
    a.E = f.E;
    a.dH = f.dH;
    a.dZ = f.dZ;
    T *dq = static_cast<T*>(f.d_q), *dk = static_cast<T*>(f.d_k), *dv = static_cast<T*>(f.d_v);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(d.B) * d.HK * d.N));
    auto run = [&](auto r) {
        constexpr int R = decltype(r)::value;
        if (d.H == d.HK)
            k_delta_grad<IO, R, false><<<grid, 64 * GW, 0, st>>>(d, a, dq, dk, dv, f.d_g, f.d_beta);
        else
            k_delta_grad<IO, R, true><<<grid, 64 * GW, 0, st>>>(d, a, dq, dk, dv, f.d_g, f.d_beta);
        return hipGetLastError();
    };
    switch (d.R) {
        case 16: return run(std::integral_constant<int, 16>{});
        case 32: return run(std::integral_constant<int, 32>{});
        case 64: return run(std::integral_constant<int, 64>{});
        case 128: return run(std::integral_constant<int, 128>{});
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_delta_grad(const DeltaShape& d, const DeltaBufs& f, hipStream_t st) {
    return d.io == 1 ? grad_io<BF16>(d, f, st) : grad_io<F32>(d, f, st);
}

}  // namespace ssd
