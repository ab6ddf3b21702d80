// The gated delta rule: chunk preparation and the scan over chunks.
//
// Per value head, with the state H [p, r] and a_t = exp(g_t):
//   e_t = v_t - a_t H_{t-1} k_t,   H_t = a_t H_{t-1} + beta_t e_t k_t^T,   y_t = scale H_t q_t.
// Over a chunk of 64 tokens with entry state H and G the inclusive cumsum of g in the chunk,
//   Ab_ts = exp(G_t - G_s) k_t.k_s (s < t),   M = (I + Ab diag(beta))^-1,
//   E = M (V - e^G (K H^T)),   U = beta E,
//   Y = scale e^G (Q H^T) + P U with P_ts = scale exp(G_t - G_s) q_t.k_s (s <= t),
//   H' = e^{G_L} H + U^T (e^{G_L - G} K).
// M is unit lower triangular and is inverted by blocks (forward substitution inside 16 x 16
// blocks, products between them): every step works on entries of M itself, so correlated
// keys, whose powers of Ab grow without bound, cost no accuracy.
//
// The backward runs the same recurrence from the right on dH (the gradient of the state that
// leaves a chunk), with N = (I + diag(beta) Ab)^-1 = I - diag(beta) M Ab:
//   dU = P^T dY + e^{G_L - G} (K dH^T),   dZ = N^T dU,   dR = beta dZ (= dV),
//   dH <- e^{G_L} dH + dY^T (scale e^G Q) - dR^T (e^G K).
// It needs no state of the forward, so both recurrences run in one launch.
//
// Tokens past a row's length are zeros in every operand with g = beta = 0: they change no
// state, give zero outputs and gradients, and their memory is not read.
#include "delta_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {

namespace {

constexpr int CS = DL + 4;  // LDS row stride of a 64 x 64 fp32 matrix

// Below this a log decay counts as this: exp() of either is zero in fp32, and differences of
// cumulative sums stay finite where g is -inf (a state that is forgotten at once).
constexpr float kMinLogDecay = -1.0e4f;

__device__ __forceinline__ int chunk_tokens(const int64_t* len, int b, int S, int c) {
    const int n = (len ? static_cast<int>(len[b]) : S) - c * DL;
    return n < 0 ? 0 : (n > DL ? DL : n);
}

// One 16 x 16 tile of a product of fp32 LDS matrices (row stride CS): A rows, B columns.
__device__ __forceinline__ v4f tile_mul(const float* A, const float* B, int i, int g, v4f c) {
#pragma unroll
    for (int k = 0; k < 16; k += 4) c = mfma16(A[i * CS + k + g], B[(k + g) * CS + i], c);
    return c;
}
// The same with the right factor in result registers.
__device__ __forceinline__ v4f tile_mul(const float* A, v4f y, int i, int g, v4f c) {
    const v4f a = *reinterpret_cast<const v4f*>(A + i * CS + 4 * g);
#pragma unroll
    for (int v = 0; v < 4; ++v) c = mfma16(a[v], y[v], c);
    return c;
}
__device__ __forceinline__ void tile_store_neg(float* X, v4f y, int i, int g) {
#pragma unroll
    for (int v = 0; v < 4; ++v) X[(4 * g + v) * CS + i] = -y[v];
}

// X = (I + C)^-1 for C strictly lower triangular (tiles above the diagonal of either are
// never read or written).  256 threads; ends without a barrier.
__device__ __forceinline__ void invert_lower(const float* C, float* X) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    const int d = 16 * w * CS + 16 * w;
    {  // diagonal blocks: lane i solves column i
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float acc = t == i ? 1.0f : 0.0f;
#pragma unroll
            for (int s = 0; s < t; ++s) acc -= C[d + t * CS + s] * x[s];
            x[t] = acc;
        }
        if (g == 0) {
#pragma unroll
            for (int t = 0; t < 16; ++t) X[d + t * CS + i] = x[t];
        }
    }
    __syncthreads();
    auto at = [](int a, int b) { return 16 * a * CS + 16 * b; };
    if (w < 2) {  // (1, 0) and (3, 2): -X_hi C X_lo
        const int lo = 2 * w, hi = 2 * w + 1;
        const v4f y = tile_mul(C + at(hi, lo), X + at(lo, lo), i, g, zero4());
        tile_store_neg(X + at(hi, lo), tile_mul(X + at(hi, hi), y, i, g, zero4()), i, g);
    }
    __syncthreads();
    {  // the 32 x 32 block below the diagonal: wave w has tile (2 + w / 2, w % 2)
        const int b = w & 1, a = 2 + (w >> 1);
        auto col = [&](int row) {
            v4f y = tile_mul(C + at(row, 1), X + at(1, b), i, g, zero4());
            if (b == 0) y = tile_mul(C + at(row, 0), X + at(0, 0), i, g, y);
            return y;
        };
        v4f x = tile_mul(X + at(a, 2), col(2), i, g, zero4());
        if (a == 3) x = tile_mul(X + at(3, 3), col(3), i, g, x);
        tile_store_neg(X + at(a, b), x, i, g);
    }
}

}  // namespace

// Per (b, h, chunk): the chunk's decay factors (coef: e^G, e^{G_L - G}, beta, and G in base 2
// and fp64) and its
// triangular matrices as bf16 parts in operand order.  Forward: M and P (rows t, k over s);
// backward: M, and N^T and P^T (rows s, k over t).
template <class IO, int R, bool BWD>
__global__ __launch_bounds__(256) void k_delta_prep(DeltaShape d, const typename IO::T* __restrict__ q,
                                                    const typename IO::T* __restrict__ k,
                                                    const float* __restrict__ gate,
                                                    const float* __restrict__ beta,
                                                    const int64_t* __restrict__ len,
                                                    float* __restrict__ coef, uint16_t* __restrict__ Mo,
                                                    uint16_t* __restrict__ Po, uint16_t* __restrict__ No) {
    constexpr int NP = in_parts<IO>(), KJ = R < 32 ? 1 : R / 32;
    constexpr int NY = BWD ? 3 : (NP == 1 ? 2 : 3);
    __shared__ double sG[DL];
    __shared__ float sBeta[DL];
    __shared__ __align__(16) float sC[DL * CS];
    __shared__ __align__(16) float sX[DL * CS];
    __shared__ __align__(16) float sAb[BWD ? DL * CS : 4];
    const int64_t ch = blockIdx.x;
    const int c = static_cast<int>(ch % d.N);
    const int64_t bh = ch / d.N;
    const int h = static_cast<int>(bh % d.H), b = static_cast<int>(bh / d.H);
    const int L = chunk_tokens(len, b, d.S, c);
    if (L == 0) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    const int64_t t0 = static_cast<int64_t>(c) * DL;
    if (w == 0) {
        const int64_t at = (static_cast<int64_t>(b) * d.S + t0 + lane) * d.H + h;
        const float gv = lane < L ? gate[at] : 0.0f;
        const float bv = lane < L ? beta[at] : 0.0f;
        double G = gv < kMinLogDecay ? kMinLogDecay : gv;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double u = __shfl_up(G, o);
            if (lane >= o) G += u;
        }
        const double G2 = G * kLog2e, tot = __shfl(G2, 63);
        sG[lane] = G2;
        sBeta[lane] = bv;
        float* cf = coef + ch * DCOEF;
        cf[lane] = exp2_of(G2);
        cf[DL + lane] = exp2_of(tot - G2);
        cf[2 * DL + lane] = bv;
        reinterpret_cast<double*>(cf + 3 * DL)[lane] = G2;
    }
    const int hk = h / (d.H / d.HK);
    const typename IO::T* kb = k + b * d.ks[0] + t0 * d.ks[1] + hk * d.ks[2];
    const typename IO::T* qb = q + b * d.qs[0] + t0 * d.qs[1] + hk * d.qs[2];
    auto row = [&](const typename IO::T* base, int64_t stride, int tile, int j) {
        const int t = 16 * tile + i, col = 32 * j + 8 * g;
        return load_parts8<IO>(base + t * stride + col, t < L && (R >= 32 || col < R));
    };
    // wave w: row tile w of K K^T and Q K^T as D[s][t] (lane t = 16 w + i, s = 16 sg + 4 g + v),
    // or for the backward Q K^T as D[t][s] (lane s = 16 w + i)
    v4f kk[4], qk[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) kk[s] = qk[s] = zero4();
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
        const auto kw = row(kb, d.ks[1], w, j);
        const auto qw = row(qb, d.qs[1], w, j);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s <= w) {
                const auto ks = row(kb, d.ks[1], s, j);
                kk[s] = mma(ks, kw, kk[s]);
                if constexpr (!BWD) qk[s] = mma(ks, qw, qk[s]);
            }
            if constexpr (BWD) {
                if (s >= w) qk[s] = mma(row(qb, d.qs[1], s, j), kw, qk[s]);
            }
        }
    }
    __syncthreads();
    {
        const int t = 16 * w + i;
        const double Gt = sG[t];
        v4f p[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            p[s] = zero4();
            if (s <= w) {
                v4f cc, ab;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int src = 16 * s + 4 * g + v;
                    const float e = exp2_of(src <= t ? Gt - sG[src] : 0.0);
                    ab[v] = src < t ? kk[s][v] * e : 0.0f;
                    cc[v] = ab[v] * sBeta[src];
                    if constexpr (!BWD) p[s][v] = src <= t ? d.scale * qk[s][v] * e : 0.0f;
                }
                *reinterpret_cast<v4f*>(sC + t * CS + 16 * s + 4 * g) = cc;
                if constexpr (BWD) *reinterpret_cast<v4f*>(sAb + t * CS + 16 * s + 4 * g) = ab;
            }
            if constexpr (BWD) {
                if (s >= w) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int tt = 16 * s + 4 * g + v;  // lane's token t is the source here
                        p[s][v] = tt >= t ? d.scale * qk[s][v] * exp2_of(sG[tt] - Gt) : 0.0f;
                    }
                }
            }
        }
        uint16_t* po = Po + ch * (NY * DTRI * DTILE);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (BWD ? j >= w / 2 : j <= w / 2) {
                const auto pp = split44<NY>(p[2 * j], p[2 * j + 1]);
                const int tile = BWD ? tri_upper(w, j) : tri_lower(w, j);
#pragma unroll
                for (int n = 0; n < NY; ++n)
                    *reinterpret_cast<b8v*>(po + (n * DTRI + tile) * DTILE + lane * 8) = pp.p[n];
            }
        }
    }
    __syncthreads();
    invert_lower(sC, sX);
    __syncthreads();
    uint16_t* mo = Mo + ch * (3 * DTRI * DTILE);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (j <= w / 2) {
            v4f m[2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                m[hf] = 2 * j + hf <= w
                            ? *reinterpret_cast<const v4f*>(sX + (16 * w + i) * CS + 32 * j + 16 * hf + 4 * g)
                            : zero4();
            const auto mp = split44<3>(m[0], m[1]);
#pragma unroll
            for (int n = 0; n < 3; ++n)
                *reinterpret_cast<b8v*>(mo + (n * DTRI + tri_lower(w, j)) * DTILE + lane * 8) = mp.p[n];
        }
    }
    if constexpr (BWD) {
        uint16_t* no = No + ch * (3 * DTRI * DTILE);
        v4f nt[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            nt[a] = zero4();
            if (a >= w) {
                v4f y = zero4();
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (u >= w && u <= a)
                        y = tile_mul(sX + 16 * a * CS + 16 * u, sAb + 16 * u * CS + 16 * w, i, g, y);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int t = 16 * a + 4 * g + v;
                    nt[a][v] = (t == 16 * w + i ? 1.0f : 0.0f) - sBeta[t] * y[v];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (j >= w / 2) {
                const auto np = split44<3>(nt[2 * j], nt[2 * j + 1]);
#pragma unroll
                for (int n = 0; n < 3; ++n)
                    *reinterpret_cast<b8v*>(no + (n * DTRI + tri_upper(w, j)) * DTILE + lane * 8) = np.p[n];
            }
        }
    }
}

namespace {

// Shared memory of one scan workgroup.
template <class IO, int R, int NQ>
struct ScanLds {
    static constexpr int NP = in_parts<IO>(), RP = R < 32 ? 32 : R, LD = RP + 8;
    uint16_t K[NP][DL * LD];
    uint16_t Q[NQ ? NP : 1][NQ ? DL * LD : 8];
    uint16_t M[3][DTRI * DTILE];
    uint16_t P[NQ ? NQ : 1][NQ ? DTRI * DTILE : 8];
    float cf[3 * DL];  // e^G, e^{G_L - G}, beta
};

// Rows [0, L) of a chunk's keys or queries as bf16 parts, zeros elsewhere.
template <class IO, int R, int NTHR>
__device__ __forceinline__ void stage_parts(uint16_t* dst, int part_stride, const typename IO::T* src,
                                            int64_t stride, int L) {
    constexpr int RP = R < 32 ? 32 : R, V = RP / 8;
#pragma unroll 4
    for (int idx = threadIdx.x; idx < DL * V; idx += NTHR) {
        const int t = idx / V, col = 8 * (idx % V);
        const auto p = load_parts8<IO>(src + t * stride + col, t < L && col < R);
#pragma unroll
        for (int n = 0; n < in_parts<IO>(); ++n)
            *reinterpret_cast<b8v*>(dst + n * part_stride + t * (RP + 8) + col) = p.p[n];
    }
}
template <int N16, int NTHR>
__device__ __forceinline__ void stage_copy(uint16_t* dst, const uint16_t* src) {
#pragma unroll 4
    for (int idx = threadIdx.x; idx < N16 / 8; idx += NTHR)
        reinterpret_cast<uint4*>(dst)[idx] = reinterpret_cast<const uint4*>(src)[idx];
}

// A operand: rows t = 16 tau + i of a staged matrix, k = 32 j + 8 g ...
template <int NP, int LD>
__device__ __forceinline__ Parts<NP> row_op(const uint16_t (*m)[DL * LD], int tau, int j, int i, int g) {
    Parts<NP> o;
#pragma unroll
    for (int n = 0; n < NP; ++n)
        o.p[n] = *reinterpret_cast<const b8v*>(&m[n][(16 * tau + i) * LD + 32 * j + 8 * g]);
    return o;
}
// A operand: the transposed matrix, rows r = 32 (tau / 2) + 8 (i / 4) + 4 (tau % 2) + i % 4 and
// k over the tokens 32 j + {4 g + v, 16 + 4 g + v}: result row 4 g + v of state tile tau is
// then r = 32 (tau / 2) + 8 g + 4 (tau % 2) + v, so that two state tiles hold eight
// consecutive r per lane.
template <int NP, int LD>
__device__ __forceinline__ Parts<NP> col_op(const uint16_t (*m)[DL * LD], int tau, int j, int i, int g) {
    Parts<NP> o;
    const int at = (32 * j + 4 * g + (i >> 2)) * LD + 32 * (tau >> 1) + 8 * (i & 3) + 4 * (tau & 1);
#pragma unroll
    for (int n = 0; n < NP; ++n) o.p[n] = join8(lds_col4(&m[n][at]), lds_col4(&m[n][at + 16 * LD]));
    return o;
}
template <int N>
__device__ __forceinline__ Parts<N> tri_op(const uint16_t (*m)[DTRI * DTILE], int tile, int lane) {
    Parts<N> o;
#pragma unroll
    for (int n = 0; n < N; ++n) o.p[n] = *reinterpret_cast<const b8v*>(&m[n][tile * DTILE + lane * 8]);
    return o;
}

template <class IO>
__device__ __forceinline__ float load_or0(const typename IO::T* p, bool on) {
    return on ? io<IO>::ld(p, 0) : 0.0f;
}

// State tiles of one wave (16 value rows p, lane i; all r) from / to [p, r] rows.
template <int R, int RT>
__device__ __forceinline__ void load_state(v4f (&s)[RT], const float* src, int i, int g) {
#pragma unroll
    for (int tau = 0; tau < RT; ++tau) {
        const int r = 32 * (tau >> 1) + 8 * g + 4 * (tau & 1);
        s[tau] = src && r < R ? *reinterpret_cast<const v4f*>(src + i * R + r) : zero4();
    }
}
template <int R, int RT>
__device__ __forceinline__ void store_state(const v4f (&s)[RT], float* dst, int i, int g) {
#pragma unroll
    for (int tau = 0; tau < RT; ++tau) {
        const int r = 32 * (tau >> 1) + 8 * g + 4 * (tau & 1);
        if (r < R) *reinterpret_cast<v4f*>(dst + i * R + r) = s[tau];
    }
}
// ... and to the [r, P] rows that the gradient kernel reads (dst at the wave's first p).
template <int R, int RT>
__device__ __forceinline__ void store_state_t(const v4f (&s)[RT], float* dst, int P, int i, int g) {
#pragma unroll
    for (int tau = 0; tau < RT; ++tau) {
        const int r = 32 * (tau >> 1) + 8 * g + 4 * (tau & 1);
        if (r < R) {
#pragma unroll
            for (int v = 0; v < 4; ++v) dst[(r + v) * P + i] = s[tau][v];
        }
    }
}

// The forward recurrence of one workgroup: W waves, each 16 value rows.  NQ > 0: the outputs,
// with y's intra-chunk operands in NQ parts; NQ = 0: the entry states and E for the backward.
template <class IO, int R, int W, int NQ>
__device__ void scan_fwd(ScanLds<IO, R, NQ>& sm, const DeltaShape& d, const DeltaScan<typename IO::T>& a,
                         int64_t blk) {
    using LDS = ScanLds<IO, R, NQ>;
    constexpr int NP = LDS::NP, RP = LDS::RP, LD = LDS::LD, KJ = RP / 32, RT = RP / 16, NTHR = 64 * W;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    const int pbs = d.P / (16 * W);
    const int p0 = static_cast<int>(blk % pbs) * 16 * W + 16 * w;
    const int64_t bh = blk / pbs;
    const int h = static_cast<int>(bh % d.H), b = static_cast<int>(bh / d.H);
    const int hk = h / (d.H / d.HK);
    const int64_t state_at = (bh * d.P + p0) * R;
    v4f s[RT];
    load_state<R>(s, a.init ? a.init + state_at : nullptr, i, g);
    int c = 0;
    for (; c < d.N; ++c) {
        const int L = chunk_tokens(a.len, b, d.S, c);
        if (L == 0) break;
        const int64_t ch = bh * d.N + c, t0 = static_cast<int64_t>(c) * DL;
        __syncthreads();
        stage_parts<IO, R, NTHR>(sm.K[0], DL * LD, a.k + b * d.ks[0] + t0 * d.ks[1] + hk * d.ks[2], d.ks[1], L);
        stage_copy<3 * DTRI * DTILE, NTHR>(sm.M[0], a.M + ch * (3 * DTRI * DTILE));
        if constexpr (NQ > 0) {
            stage_parts<IO, R, NTHR>(sm.Q[0], DL * LD, a.q + b * d.qs[0] + t0 * d.qs[1] + hk * d.qs[2], d.qs[1], L);
            stage_copy<NQ * DTRI * DTILE, NTHR>(sm.P[0], a.P + ch * (NQ * DTRI * DTILE));
        }
        for (int idx = threadIdx.x; idx < 3 * DL; idx += NTHR) sm.cf[idx] = a.coef[ch * DCOEF + idx];
        __syncthreads();
        v4f x[4], y[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = y[t] = zero4();
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            const auto sp = split44<3>(s[2 * j], s[2 * j + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = mma(row_op<NP, LD>(sm.K, t, j, i, g), sp, x[t]);
            if constexpr (NQ > 0) {
                Parts<NQ> sy;
#pragma unroll
                for (int n = 0; n < NQ; ++n) sy.p[n] = sp.p[n];
#pragma unroll
                for (int t = 0; t < 4; ++t) y[t] = mma(sy, row_op<NP, LD>(sm.Q, t, j, i, g), y[t]);
            }
        }
        // R = V - e^G X, E = M R, U = beta E (lane: value row p0 + i, tokens 16 tau + 4 g + v)
        v4f rr[4], u[4];
        const typename IO::T* vb = a.v + b * d.vs[0] + t0 * d.vs[1] + h * d.vs[2] + p0 + i;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const v4f eg = *reinterpret_cast<const v4f*>(&sm.cf[16 * t + 4 * g]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int tok = 16 * t + 4 * g + v;
                rr[t][v] = load_or0<IO>(vb + tok * d.vs[1], tok < L) - eg[v] * x[t][v];
            }
            u[t] = zero4();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const auto rp = split44<3>(rr[2 * j], rr[2 * j + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (j <= t / 2) u[t] = mma(tri_op<3>(sm.M, tri_lower(t, j), lane), rp, u[t]);
        }
        if constexpr (NQ == 0) {
            store_state_t<R>(s, a.H + ch * (R * d.P) + p0, d.P, i, g);
            float* eo = a.E + ch * (DL * d.P) + p0 + i;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int v = 0; v < 4; ++v) eo[(16 * t + 4 * g + v) * d.P] = u[t][v];
        }
        v4f ut[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            u[t] *= *reinterpret_cast<const v4f*>(&sm.cf[2 * DL + 16 * t + 4 * g]);
            ut[t] = u[t] * *reinterpret_cast<const v4f*>(&sm.cf[DL + 16 * t + 4 * g]);
        }
        const float eL = sm.cf[DL - 1];
#pragma unroll
        for (int t = 0; t < RT; ++t) s[t] *= eL;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const auto up = split44<3>(ut[2 * j], ut[2 * j + 1]);
#pragma unroll
            for (int t = 0; t < RT; ++t) s[t] = mma(col_op<NP, LD>(sm.K, t, j, i, g), up, s[t]);
        }
        if constexpr (NQ > 0) {
#pragma unroll
            for (int t = 0; t < 4; ++t) y[t] *= d.scale * sm.cf[16 * t + i];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const auto up = split44<NQ>(u[2 * j], u[2 * j + 1]);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (j <= t / 2) y[t] = mma(up, tri_op<NQ>(sm.P, tri_lower(t, j), lane), y[t]);
            }
            // y holds D[p][t]: lane token 16 tau + i, value rows 4 g + v
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t tok = t0 + 16 * t + i;
                if (tok < d.S) io<IO>::st4(a.y, ((b * static_cast<int64_t>(d.S) + tok) * d.H + h) * d.P + p0 + 4 * g, y[t]);
            }
        }
        mfma_settle();
    }
    if (a.final_state) store_state<R>(s, a.final_state + state_at, i, g);
    if constexpr (NQ > 0) {  // chunks past the row's length
        for (int64_t tok = static_cast<int64_t>(c) * DL + i; tok < d.S; tok += 16)
            io<IO>::st4(a.y, ((b * static_cast<int64_t>(d.S) + tok) * d.H + h) * d.P + p0 + 4 * g, zero4());
    }
}

// The reverse recurrence: writes the gradient of the state leaving each chunk and dZ.
template <class IO, int R, int W>
__device__ void scan_rev(ScanLds<IO, R, 3>& sm, const DeltaShape& d, const DeltaScan<typename IO::T>& a,
                         int64_t blk) {
    using LDS = ScanLds<IO, R, 3>;
    constexpr int NP = LDS::NP, RP = LDS::RP, LD = LDS::LD, KJ = RP / 32, RT = RP / 16, NTHR = 64 * W;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    const int pbs = d.P / (16 * W);
    const int p0 = static_cast<int>(blk % pbs) * 16 * W + 16 * w;
    const int64_t bh = blk / pbs;
    const int h = static_cast<int>(bh % d.H), b = static_cast<int>(bh / d.H);
    const int hk = h / (d.H / d.HK);
    const int64_t state_at = (bh * d.P + p0) * R;
    v4f s[RT];
    load_state<R>(s, a.d_final ? a.d_final + state_at : nullptr, i, g);
    for (int c = d.N - 1; c >= 0; --c) {
        const int L = chunk_tokens(a.len, b, d.S, c);
        if (L == 0) continue;
        const int64_t ch = bh * d.N + c, t0 = static_cast<int64_t>(c) * DL;
        __syncthreads();
        stage_parts<IO, R, NTHR>(sm.K[0], DL * LD, a.k + b * d.ks[0] + t0 * d.ks[1] + hk * d.ks[2], d.ks[1], L);
        stage_parts<IO, R, NTHR>(sm.Q[0], DL * LD, a.q + b * d.qs[0] + t0 * d.qs[1] + hk * d.qs[2], d.qs[1], L);
        stage_copy<3 * DTRI * DTILE, NTHR>(sm.M[0], a.NT + ch * (3 * DTRI * DTILE));
        stage_copy<3 * DTRI * DTILE, NTHR>(sm.P[0], a.P + ch * (3 * DTRI * DTILE));
        for (int idx = threadIdx.x; idx < 3 * DL; idx += NTHR) sm.cf[idx] = a.coef[ch * DCOEF + idx];
        store_state_t<R>(s, a.dH + ch * (R * d.P) + p0, d.P, i, g);
        __syncthreads();
        v4f x[4], dy[4];
        const typename IO::T* yb = a.dy + ((b * static_cast<int64_t>(d.S) + t0) * d.H + h) * d.P + p0 + i;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            x[t] = zero4();
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int tok = 16 * t + 4 * g + v;
                dy[t][v] = load_or0<IO>(yb + static_cast<int64_t>(tok) * d.H * d.P, tok < L);
            }
        }
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            const auto sp = split44<3>(s[2 * j], s[2 * j + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = mma(row_op<NP, LD>(sm.K, t, j, i, g), sp, x[t]);
        }
        v4f z[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            x[t] *= *reinterpret_cast<const v4f*>(&sm.cf[DL + 16 * t + 4 * g]);
            z[t] = zero4();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const auto yp = split44<NP>(dy[2 * j], dy[2 * j + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (j >= t / 2) x[t] = mma(tri_op<3>(sm.P, tri_upper(t, j), lane), yp, x[t]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const auto up = split44<3>(x[2 * j], x[2 * j + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (j >= t / 2) z[t] = mma(tri_op<3>(sm.M, tri_upper(t, j), lane), up, z[t]);
        }
        float* zo = a.dZ + ch * (DL * d.P) + p0 + i;
        const float eL = sm.cf[DL - 1];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const v4f eg = *reinterpret_cast<const v4f*>(&sm.cf[16 * t + 4 * g]);
            const v4f be = *reinterpret_cast<const v4f*>(&sm.cf[2 * DL + 16 * t + 4 * g]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                zo[(16 * t + 4 * g + v) * d.P] = z[t][v];
                z[t][v] *= -eg[v] * be[v];
                dy[t][v] *= d.scale * eg[v];
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) s[t] *= eL;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const auto zp = split44<3>(z[2 * j], z[2 * j + 1]);
            const auto yp = split44<3>(dy[2 * j], dy[2 * j + 1]);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                s[t] = mma(col_op<NP, LD>(sm.K, t, j, i, g), zp, s[t]);
                s[t] = mma(col_op<NP, LD>(sm.Q, t, j, i, g), yp, s[t]);
            }
        }
        mfma_settle();
    }
    if (a.d_init) store_state<R>(s, a.d_init + state_at, i, g);
}

}  // namespace

template <class IO, int R, int W>
__global__ __launch_bounds__(64 * W) void k_delta_scan(DeltaShape d, DeltaScan<typename IO::T> a) {
    constexpr int NQ = in_parts<IO>() == 1 ? 2 : 3;
    __shared__ __align__(16) ScanLds<IO, R, NQ> sm;
    scan_fwd<IO, R, W, NQ>(sm, d, a, blockIdx.x);
}

// Both recurrences of the backward: the first half of the grid recomputes the entry states,
// the second half runs the reverse.
template <class IO, int R, int W>
__global__ __launch_bounds__(64 * W) void k_delta_states(DeltaShape d, DeltaScan<typename IO::T> a) {
    __shared__ __align__(16) union Lds {
        ScanLds<IO, R, 0> f;
        ScanLds<IO, R, 3> r;
    } sm;
    const int64_t half = gridDim.x / 2;
    if (blockIdx.x < half)
        scan_fwd<IO, R, W, 0>(sm.f, d, a, blockIdx.x);
    else
        scan_rev<IO, R, W>(sm.r, d, a, blockIdx.x - half);
}

namespace {

template <class IO>
DeltaScan<typename IO::T> typed(const DeltaBufs& f) {
    using T = typename IO::T;
    DeltaScan<T> a;
    a.q = static_cast<const T*>(f.q);
    a.k = static_cast<const T*>(f.k);
    a.v = static_cast<const T*>(f.v);
    a.dy = static_cast<const T*>(f.dy);
    a.y = static_cast<T*>(f.y);
    a.len = f.len;
    a.init = f.init;
    a.d_final = f.d_final;
    a.final_state = f.final_state;
    a.d_init = f.d_init;
    a.coef = f.coef;
    a.M = f.M;
    a.P = f.P;
    a.NT = f.NT;
    a.H = f.H;
    a.E = f.E;
    a.dH = f.dH;
    a.dZ = f.dZ;
    return a;
}

template <class IO, int R>
hipError_t prep_r(const DeltaShape& d, const DeltaBufs& f, bool bwd, hipStream_t st) {
    const auto a = typed<IO>(f);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(d.B) * d.H * d.N));
    if (bwd)
        k_delta_prep<IO, R, true><<<grid, 256, 0, st>>>(d, a.q, a.k, f.g, f.beta, a.len, a.coef, a.M, a.P, a.NT);
    else
        k_delta_prep<IO, R, false><<<grid, 256, 0, st>>>(d, a.q, a.k, f.g, f.beta, a.len, a.coef, a.M, a.P, nullptr);
    return hipGetLastError();
}

template <class IO, int R, int W>
hipError_t scan_w(const DeltaShape& d, const DeltaBufs& f, bool bwd, hipStream_t st) {
    const auto a = typed<IO>(f);
    const int64_t wgs = static_cast<int64_t>(d.B) * d.H * (d.P / (16 * W));
    if (bwd)
        k_delta_states<IO, R, W><<<dim3(static_cast<unsigned>(2 * wgs)), 64 * W, 0, st>>>(d, a);
    else
        k_delta_scan<IO, R, W><<<dim3(static_cast<unsigned>(wgs)), 64 * W, 0, st>>>(d, a);
    return hipGetLastError();
}

template <class IO, int R>
hipError_t scan_r(const DeltaShape& d, const DeltaBufs& f, bool bwd, hipStream_t st) {
    switch (d.P) {
        case 16: return scan_w<IO, R, 1>(d, f, bwd, st);
        case 32: return scan_w<IO, R, 2>(d, f, bwd, st);
        case 64:
        case 128: return scan_w<IO, R, 4>(d, f, bwd, st);
        default: return hipErrorInvalidValue;
    }
}

template <class IO>
hipError_t by_r(const DeltaShape& d, const DeltaBufs& f, bool prep, bool bwd, hipStream_t st) {
    switch (d.R) {
        case 16: return prep ? prep_r<IO, 16>(d, f, bwd, st) : scan_r<IO, 16>(d, f, bwd, st);
        case 32: return prep ? prep_r<IO, 32>(d, f, bwd, st) : scan_r<IO, 32>(d, f, bwd, st);
        case 64: return prep ? prep_r<IO, 64>(d, f, bwd, st) : scan_r<IO, 64>(d, f, bwd, st);
        case 128: return prep ? prep_r<IO, 128>(d, f, bwd, st) : scan_r<IO, 128>(d, f, bwd, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_delta_prep(const DeltaShape& d, const DeltaBufs& f, bool bwd, hipStream_t st) {
    return d.io == 1 ? by_r<BF16>(d, f, true, bwd, st) : by_r<F32>(d, f, true, bwd, st);
}

hipError_t launch_delta_scan(const DeltaShape& d, const DeltaBufs& f, bool bwd, hipStream_t st) {
    return d.io == 1 ? by_r<BF16>(d, f, false, bwd, st) : by_r<F32>(d, f, false, bwd, st);
}

}  // namespace ssd
