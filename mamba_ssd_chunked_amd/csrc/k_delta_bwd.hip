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
// head are added up in its registers, in order.  Value columns go through LDS 32 at a time; a
// wave owns one 16-row tile of r and its tiles of tokens, so H and dH are read once, straight
// into operand registers.
#include "delta_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {

namespace {

constexpr int PB = 32;       // value columns staged at a time
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

template <class IO, int R>
__global__ __launch_bounds__(512) void k_delta_grad(DeltaShape d, DeltaScan<typename IO::T> a,
                                                    typename IO::T* __restrict__ d_q,
                                                    typename IO::T* __restrict__ d_k,
                                                    typename IO::T* __restrict__ d_v,
                                                    float* __restrict__ d_g, float* __restrict__ d_beta) {
    using T = typename IO::T;
    constexpr int NP = in_parts<IO>(), RP = R < 32 ? 32 : R, LD = RP + 8, KJ = RP / 32;
    constexpr int RT = R / 16, ITEMS = RT < 2 ? 1 : RT / 2, V = RP / 8;
    constexpr int KQ = DL * LD, UP = DL * LP, SP = DL * LS;
    __shared__ __align__(16) uint16_t sK[NP * KQ], sQ[NP * KQ];
    __shared__ __align__(16) union {
        struct {
            uint16_t U[3 * UP], Z[3 * UP], Y[NP * UP];
        } v;
        uint16_t S[3 * SP];
    } sm;
    __shared__ float sCf[3 * DL + 1];  // e^G, e^{G_L - G}, beta, e^{G_L}
    __shared__ double sG[DL];
    __shared__ float sLoc[RT][DL], sWr[RT][DL], sRow[4][DL], sCol[4][DL], sDot[8];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, i = lane & 15, g = lane >> 4;
    const int64_t blk = blockIdx.x;
    const int c = static_cast<int>(blk % d.N);
    const int hk = static_cast<int>((blk / d.N) % d.HK), b = static_cast<int>(blk / d.N / d.HK);
    const int64_t t0 = static_cast<int64_t>(c) * DL;
    const int grp = d.H / d.HK;
    const int all = static_cast<int>(d.S - t0 < DL ? d.S - t0 : DL);  // rows of the tensors
    int64_t n = (a.len ? a.len[b] : d.S) - t0;
    const int L = n < 0 ? 0 : (n > DL ? DL : static_cast<int>(n));
    const int64_t row0 = static_cast<int64_t>(b) * d.S + t0;
    if (L == 0) {  // past the row's length
        for (int idx = tid; idx < all * (R / 4); idx += 512) {
            const int64_t at = ((row0 + idx / (R / 4)) * d.HK + hk) * R + 4 * (idx % (R / 4));
            io<IO>::st4(d_q, at, zero4());
            io<IO>::st4(d_k, at, zero4());
        }
        for (int hh = 0; hh < grp; ++hh) {
            const int h = hk * grp + hh;
            for (int idx = tid; idx < all * (d.P / 4); idx += 512)
                io<IO>::st4(d_v, ((row0 + idx / (d.P / 4)) * d.H + h) * d.P + 4 * (idx % (d.P / 4)), zero4());
            if (tid < all) d_g[(row0 + tid) * d.H + h] = d_beta[(row0 + tid) * d.H + h] = 0.0f;
        }
        return;
    }
    {
        const T* kb = a.k + b * d.ks[0] + t0 * d.ks[1] + hk * d.ks[2];
        const T* qb = a.q + b * d.qs[0] + t0 * d.qs[1] + hk * d.qs[2];
        for (int idx = tid; idx < DL * V; idx += 512) {
            const int t = idx / V, col = 8 * (idx % V);
            const bool on = t < L && col < R;
            const auto kp = load_parts8<IO>(kb + t * d.ks[1] + col, on);
            const auto qp = load_parts8<IO>(qb + t * d.qs[1] + col, on);
#pragma unroll
            for (int m = 0; m < NP; ++m) {
                *reinterpret_cast<b8v*>(sK + m * KQ + t * LD + col) = kp.p[m];
                *reinterpret_cast<b8v*>(sQ + m * KQ + t * LD + col) = qp.p[m];
            }
        }
    }
    const int rho = w * ITEMS / 4, tt0 = (w * ITEMS) & 3;  // this wave's r tile and first token tile
    const bool act = rho < RT;
    v4f dq[ITEMS], dk[ITEMS];
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) dq[m] = dk[m] = zero4();
    // the causal pair tiles (token tile tau, source tile sigma) of this wave: w and w + 8 of ten
    auto tau_of = [](int idx) { return idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3; };
    const int ntile = w < 2 ? 2 : 1;

    for (int hh = 0; hh < grp; ++hh) {
        const int h = hk * grp + hh;
        const int64_t ch = (static_cast<int64_t>(b) * d.H + h) * d.N + c;
        const float* cf = a.coef + ch * DCOEF;
        __syncthreads();
        if (tid <= 3 * DL) sCf[tid] = cf[tid];
        if (tid < DL) sG[tid] = reinterpret_cast<const double*>(cf + DCF)[tid];
        v4f aq[ITEMS], akr[ITEMS], akw[ITEMS], dP[2], dA[2];
#pragma unroll
        for (int m = 0; m < ITEMS; ++m) aq[m] = akr[m] = akw[m] = zero4();
        dP[0] = dP[1] = dA[0] = dA[1] = zero4();
        float db = 0.0f, hdh = 0.0f;
        const float* Hc = a.H + ch * (static_cast<int64_t>(R) * d.P);
        const float* dHc = a.dH + ch * (static_cast<int64_t>(R) * d.P);
        const float* Ec = a.E + ch * (static_cast<int64_t>(DL) * d.P);
        const float* Zc = a.dZ + ch * (static_cast<int64_t>(DL) * d.P);
        for (int p0 = 0; p0 < d.P; p0 += PB) {
            __syncthreads();
            {
                const int t = tid >> 3, pc = 4 * (tid & 7), p = p0 + pc;
                v4f e = zero4(), z = zero4(), y = zero4();
                if (p < d.P) {
                    e = *reinterpret_cast<const v4f*>(Ec + t * d.P + p);
                    z = *reinterpret_cast<const v4f*>(Zc + t * d.P + p);
                    if (t < L) y = io<IO>::ld4(a.dy, ((row0 + t) * d.H + h) * d.P + p);
                }
                const float be = sCf[2 * DL + t];
                db += e[0] * z[0] + e[1] * z[1] + e[2] * z[2] + e[3] * z[3];
                e *= be;
                z *= be;
                if (p < d.P && t < all) io<IO>::st4(d_v, ((row0 + t) * d.H + h) * d.P + p, z);
                store_parts4<3>(sm.v.U + t * LP + pc, UP, e);
                store_parts4<3>(sm.v.Z + t * LP + pc, UP, z);
                store_parts4<NP>(sm.v.Y + t * LP + pc, UP, y);
            }
            Parts<3> hp, gp;
            if (act) {
                const int p = p0 + 8 * g;
                v4f h0 = zero4(), h1 = zero4(), g0 = zero4(), g1 = zero4();
                if (p < d.P) {
                    const int64_t at = static_cast<int64_t>(16 * rho + i) * d.P + p;
                    h0 = *reinterpret_cast<const v4f*>(Hc + at);
                    h1 = *reinterpret_cast<const v4f*>(Hc + at + 4);
                    g0 = *reinterpret_cast<const v4f*>(dHc + at);
                    g1 = *reinterpret_cast<const v4f*>(dHc + at + 4);
                }
                if (tt0 == 0) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) hdh += h0[v] * g0[v] + h1[v] * g1[v];
                }
                hp = split44<3>(h0, h1);
                gp = split44<3>(g0, g1);
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
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (m < ntile) {
                    const int idx = w + 8 * m, tau = tau_of(idx), sig = idx - tau * (tau + 1) / 2;
                    const auto u = rows8<3>(sm.v.U, UP, LP, 16 * sig + i, 8 * g);
                    dP[m] = mma(u, rows8<NP>(sm.v.Y, UP, LP, 16 * tau + i, 8 * g), dP[m]);
                    dA[m] = mma(u, rows8<3>(sm.v.Z, UP, LP, 16 * tau + i, 8 * g), dA[m]);
                }
            }
        }
        // results D[r][t] (lane token 16 tt + i, rows r = 16 rho + 4 g + v)
        if (act) {
#pragma unroll
            for (int m = 0; m < ITEMS; ++m) {
                const int t = 16 * (tt0 + m) + i, at = t * LD + 16 * rho + 4 * g;
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
                dq[m] += aq[m];
                dk[m] += akr[m] + akw[m];
            }
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) hdh += __shfl_xor(hdh, o);
        if (lane == 0) sDot[w] = hdh;
        // pair tiles D[s][t] (lane token 16 tau + i, sources 16 sig + 4 g + v)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (m < ntile) {
                const int idx = w + 8 * m, tau = tau_of(idx), sig = idx - tau * (tau + 1) / 2;
                v4f kk = zero4(), qk = zero4();
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    const auto ks = rows8<NP>(sK, KQ, LD, 16 * sig + i, 32 * j + 8 * g);
                    kk = mma(ks, rows8<NP>(sK, KQ, LD, 16 * tau + i, 32 * j + 8 * g), kk);
                    qk = mma(ks, rows8<NP>(sQ, KQ, LD, 16 * tau + i, 32 * j + 8 * g), qk);
                }
                const int t = 16 * tau + i;
                float wrow = 0.0f;
                v4f wcol;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int s = 16 * sig + 4 * g + v;
                    const float e = s <= t ? exp2_of(sG[t] - sG[s]) : 0.0f;
                    const float es = s < t ? e : 0.0f;
                    const float x = es * (d.scale * dP[m][v] * qk[v] - dA[m][v] * kk[v]);
                    wrow += x;
                    wcol[v] = x;
                    dP[m][v] *= d.scale * e;
                    dA[m][v] *= -es;
                }
                wrow = sum_over_g(wrow);
                if (g == 0) sRow[sig][t] = wrow;
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) wcol[v] += __shfl_xor(wcol[v], o);
                }
                if (i == 0) *reinterpret_cast<v4f*>(&sCol[tau][16 * sig + 4 * g]) = wcol;
            }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) db += __shfl_xor(db, o);
        if ((tid & 7) == 0 && (tid >> 3) < all) d_beta[(row0 + (tid >> 3)) * d.H + h] = (tid >> 3) < L ? db : 0.0f;
#pragma unroll
        for (int which = 0; which < 2; ++which) {  // dS, then dKK
            __syncthreads();
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (m < ntile) {
                    const int idx = w + 8 * m, tau = tau_of(idx), sig = idx - tau * (tau + 1) / 2;
                    uint16_t* at = sm.S + (16 * tau + i) * LS + 16 * sig + 4 * g;
                    store_parts4<3>(at, SP, which ? dA[m] : dP[m]);
                    if (sig == tau && (tau & 1) == 0) store_parts4<3>(at + 16, SP, zero4());
                }
            }
            __syncthreads();
            if (which == 1 && w == 0) {
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
                for (int m = 0; m < 8; ++m) hd += sDot[m];
                double suf = loc, pre = wr;
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) {
                    const double u = __shfl_down(suf, o), x = __shfl_up(pre, o);
                    if (lane + o < 64) suf += u;
                    if (lane >= o) pre += x;
                }
                pre = __shfl_up(pre, 1);
                if (lane == 0) pre = 0.0;
                const double out = suf + pre + static_cast<double>(sCf[3 * DL]) * hd;
                if (lane < all) d_g[(row0 + lane) * d.H + h] = lane < L ? static_cast<float>(out) : 0.0f;
            }
            if (act) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const auto kt = cols8<NP>(sK, KQ, LD, 32 * j, 16 * rho, i, g);
                    Parts<NP> xt;
                    if (which == 0) xt = cols8<NP>(sQ, KQ, LD, 32 * j, 16 * rho, i, g);
#pragma unroll
                    for (int m = 0; m < ITEMS; ++m) {
                        const int tt = tt0 + m;
                        if (j <= tt / 2) {
                            const auto x = rows8<3>(sm.S, SP, LS, 16 * tt + i, 32 * j + 8 * g);
                            if (which == 0) dq[m] = mma(kt, x, dq[m]);
                            else dk[m] = mma(kt, x, dk[m]);
                        }
                        if (j >= tt / 2) {
                            const auto x = cols8<3>(sm.S, SP, LS, 32 * j, 16 * tt, i, g);
                            dk[m] = mma(which == 0 ? xt : kt, x, dk[m]);
                        }
                    }
                }
            }
        }
    }
    if (act) {
#pragma unroll
        for (int m = 0; m < ITEMS; ++m) {
            const int t = 16 * (tt0 + m) + i;
            if (t < all) {
                const int64_t at = ((row0 + t) * d.HK + hk) * R + 16 * rho + 4 * g;
                io<IO>::st4(d_q, at, dq[m]);
                io<IO>::st4(d_k, at, dk[m]);
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
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(d.B) * d.HK * d.N)), block(512);
    switch (d.R) {
        case 16: k_delta_grad<IO, 16><<<grid, block, 0, st>>>(d, a, dq, dk, dv, f.d_g, f.d_beta); break;
        case 32: k_delta_grad<IO, 32><<<grid, block, 0, st>>>(d, a, dq, dk, dv, f.d_g, f.d_beta); break;
        case 64: k_delta_grad<IO, 64><<<grid, block, 0, st>>>(d, a, dq, dk, dv, f.d_g, f.d_beta); break;
        case 128: k_delta_grad<IO, 128><<<grid, block, 0, st>>>(d, a, dq, dk, dv, f.d_g, f.d_beta); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grad(const DeltaShape& d, const DeltaBufs& f, hipStream_t st) {
    return d.io == 1 ? grad_io<BF16>(d, f, st) : grad_io<F32>(d, f, st);
}

}  // namespace ssd
