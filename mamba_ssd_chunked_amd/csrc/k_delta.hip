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
#include <type_traits>

#include "delta_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {

namespace {

constexpr int CS = DL + 4;  // LDS row stride of a 64 x 64 fp32 matrix

// Whether the scans' loading waves take q and k through registers, to cut them into bf16 parts (fp32
// io) or to fill up rows shorter than an operand, rather than straight into LDS.
template <class IO, int R>
__host__ __device__ constexpr bool through_registers() { return in_parts<IO>() == 3 || R < 32; }

// Kilobytes of an operand tile of P: three bf16 parts, or for bf16 io's outputs its 512 fp32 values (a
// lane's first four, then all lanes' second), which the scan cuts into parts itself: 12 KB a chunk
// instead of 18, and the sums that make y keep all 24 bits of P.
template <class IO>
__host__ __device__ constexpr int p_kilobytes(bool bwd) { return bwd || in_parts<IO>() == 3 ? 3 : 2; }

// Below this a log decay counts as this: exp() of either is zero in fp32, and differences of
// cumulative sums stay finite where g is -inf (a state that is forgotten at once).
constexpr float kMinLogDecay = -1.0e4f;

__device__ __forceinline__ int chunk_tokens(const int64_t* len, int b, int S, int c) {
    const int n = (len ? static_cast<int>(len[b]) : S) - c * DL;
    return n < 0 ? 0 : (n > DL ? DL : n);
}

// The eight XCDs take workgroups in turn and each has its own L2: give each a consecutive run of
// the work, so that the columns and value heads that read the same keys meet in one.
__device__ __forceinline__ int64_t xcd_order(int64_t blk, int64_t n) {
    const int64_t x = blk % 8, q = n / 8, rem = n % 8;
    return x * q + (x < rem ? x : rem) + blk / 8;
}

// Half a lane's slots of an operand tile (four values) as N parts.
template <int N>
__device__ __forceinline__ void put_half(uint16_t* dst, int tile, int lane, int half, v4f x) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint2 w;
        w.x = f32x2_to_bf16x2(x[0], x[1]);
        w.y = f32x2_to_bf16x2(x[2], x[3]);
        *reinterpret_cast<uint2*>(dst + (n * DTRI + tile) * DTILE + lane * 8 + 4 * half) = w;
        if (n + 1 < N)
            x -= v4f{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
    }
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
    {  // diagonal blocks: lane i solves column i, each solved row at once taken off those below
        v4f cr[16][4];
#pragma unroll
        for (int t = 1; t < 16; ++t)
#pragma unroll
            for (int q = 0; q < (t + 3) / 4; ++q) cr[t][q] = *reinterpret_cast<const v4f*>(C + d + t * CS + 4 * q);
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) x[t] = t == i ? 1.0f : 0.0f;
#pragma unroll
        for (int s = 0; s < 15; ++s)
#pragma unroll
            for (int t = s + 1; t < 16; ++t) x[t] -= cr[t][s / 4][s % 4] * x[s];
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
// and fp64) and its triangular matrices in operand order, as bf16 parts (P of bf16 io's forward in
// fp32).  Forward: M and P (rows
// t, k over s); backward: M, and N^T and P^T (rows s, k over t).
//
// Wave w has the tokens 16 w .. + 15: their rows of K and Q stay in its registers as operands, and
// the key rows of the others come through LDS, which the fp32 matrices take over afterwards.
//
// Bound by HBM: it reads q and k and writes two triangular matrices.  160 heads of 64 chunks, bf16,
// r = 128: 0.79 GB in 137-147 us, 5.7 TB/s (with K and Q as fp32 in LDS and substitution there: 217
// us); 32 heads of 1024 chunks, fp32: 3.9 GB in 644-664 us.  A preparation of its own doubles the
// reads of q and k, but has the inverses, long chains of dependent steps, in 10,240 workgroups at once
// instead of in the 160 of the scan, each before the next chunk.
template <class IO, int R, bool BWD>
__global__ __launch_bounds__(256) void k_delta_prep(DeltaShape d, const typename IO::T* __restrict__ q,
                                                    const typename IO::T* __restrict__ k,
                                                    const float* __restrict__ gate,
                                                    const float* __restrict__ beta,
                                                    const int64_t* __restrict__ len,
                                                    float* __restrict__ coef, uint16_t* __restrict__ Mo,
                                                    uint16_t* __restrict__ Po, uint16_t* __restrict__ No) {
    using T = typename IO::T;
    constexpr int NP = in_parts<IO>(), KJ = R < 32 ? 1 : R / 32;
    constexpr int PK = p_kilobytes<IO>(BWD);
    constexpr int MAT = DL * CS;
    constexpr int KB = NP * 4 * KJ * 1024, MB = (BWD ? 3 : 2) * MAT * 4;
    __shared__ __align__(16) char sm[KB > MB ? KB : MB];
    __shared__ double sG[DL];
    __shared__ float sBeta[DL];
    float* sC = reinterpret_cast<float*>(sm);
    float* sX = sC + MAT;
    float* sAb = sX + MAT;
    const int64_t ch = xcd_order(blockIdx.x, gridDim.x);
    const int c = static_cast<int>(ch % d.N);
    const int64_t bh = ch / d.N;
    const int h = static_cast<int>(bh % d.H), b = static_cast<int>(bh / d.H);
    const int L = chunk_tokens(len, b, d.S, c);
    if (L == 0) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    const int64_t t0 = static_cast<int64_t>(c) * DL;
    const int hk = h / (d.H / d.HK);
    // this wave's rows of k and q; rows past the length are read as the last one, then zeroed
    typedef T raw8 __attribute__((ext_vector_type(8)));
    raw8 kr[KJ], qr[KJ];
    {
        const int t = 16 * w + i, row = t < L ? t : L - 1;
        const T* kb = k + b * d.ks[0] + (t0 + row) * d.ks[1] + hk * d.ks[2] + (R < 32 ? 8 * (g & 1) : 8 * g);
        const T* qb = q + b * d.qs[0] + (t0 + row) * d.qs[1] + hk * d.qs[2] + (R < 32 ? 8 * (g & 1) : 8 * g);
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            kr[j] = *reinterpret_cast<const raw8*>(kb + 32 * j);
            qr[j] = *reinterpret_cast<const raw8*>(qb + 32 * j);
        }
    }
    if (w == 0) {
        const int64_t at = (static_cast<int64_t>(b) * d.S + t0 + (lane < L ? lane : L - 1)) * d.H + h;
        const float gl = gate[at], bl = beta[at];
        const float gv = lane < L ? gl : 0.0f, bv = lane < L ? bl : 0.0f;
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
        cf[lane] = lane < L ? exp2_of(G2) : 0.0f;
        cf[DL + lane] = exp2_of(tot - G2);
        cf[2 * DL + lane] = bv;
        if (lane == 0) cf[3 * DL] = exp2_of(tot);
        reinterpret_cast<double*>(cf + DCF)[lane] = G2;
    }
    Parts<NP> kw[KJ], qw[KJ];
    const bool on = 16 * w + i < L && (R >= 32 || g < 2);
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
        kw[j] = parts_of<IO>(kr[j], on);
        qw[j] = parts_of<IO>(qr[j], on);
#pragma unroll
        for (int n = 0; n < NP; ++n)
            *reinterpret_cast<b8v*>(sm + ((n * 4 + w) * KJ + j) * 1024 + lane * 16) = kw[j].p[n];
    }
    __syncthreads();
    // K K^T as D[s][t] (lane token 16 w + i, sources 16 sg + 4 g + v), Q K^T the same way or, for
    // the backward's transposed operand, as D[t][s] (lane source 16 sg + i)
    v4f kk[4], qk[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) kk[s] = qk[s] = zero4();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s <= w) {
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                Parts<NP> ks;
#pragma unroll
                for (int n = 0; n < NP; ++n)
                    ks.p[n] = *reinterpret_cast<const b8v*>(sm + ((n * 4 + s) * KJ + j) * 1024 + lane * 16);
                kk[s] = mma(ks, kw[j], kk[s]);
                qk[s] = BWD ? mma(qw[j], ks, qk[s]) : mma(ks, qw[j], qk[s]);
            }
        }
    }
    __syncthreads();
    const int t = 16 * w + i;
    uint16_t* po = Po + ch * (PK * DTRI * DTILE);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s <= w) {
            v4f cc, ab;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int src = 16 * s + 4 * g + v;
                const float e = exp2_of(src <= t ? sG[t] - sG[src] : 0.0);
                ab[v] = src < t ? kk[s][v] * e : 0.0f;
                cc[v] = ab[v] * sBeta[src];
                if constexpr (!BWD) qk[s][v] = src <= t ? d.scale * qk[s][v] * e : 0.0f;
            }
            *reinterpret_cast<v4f*>(sC + t * CS + 16 * s + 4 * g) = cc;
            if constexpr (BWD) {
                *reinterpret_cast<v4f*>(sAb + t * CS + 16 * s + 4 * g) = ab;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int tt = 16 * w + 4 * g + v, src = 16 * s + i;
                    qk[s][v] = src <= tt ? d.scale * qk[s][v] * exp2_of(sG[tt] - sG[src]) : 0.0f;
                }
                put_half<3>(po, tri_upper(s, w / 2), lane, w & 1, qk[s]);
            }
        }
    }
    if constexpr (BWD) {
        if ((w & 1) == 0) put_half<3>(po, tri_upper(w + 1, w / 2), lane, 0, zero4());  // above the diagonal
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (j <= w / 2) {
                uint16_t* at = po + tri_lower(w, j) * DTILE + lane * 8;
                if constexpr (PK == 2) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) *reinterpret_cast<v4f*>(at + hf * DTRI * DTILE) = qk[2 * j + hf];
                } else {
                    const auto pp = split44<3>(qk[2 * j], qk[2 * j + 1]);
#pragma unroll
                    for (int n = 0; n < 3; ++n) *reinterpret_cast<b8v*>(at + n * DTRI * DTILE) = pp.p[n];
                }
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
                            ? *reinterpret_cast<const v4f*>(sX + t * CS + 32 * j + 16 * hf + 4 * g)
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
                    const int row = 16 * a + 4 * g + v;
                    nt[a][v] = (row == t ? 1.0f : 0.0f) - sBeta[row] * y[v];
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

// kOutputs: y and the final state; kCarry: what a segment does to the state; kRecord and kReverse: the
// backward's two recurrences.
enum ScanMode { kOutputs, kCarry, kRecord, kReverse };

// Loading waves of a scan workgroup: a wave has at most 63 loads under way, and a chunk of fp32
// operands is twice that.
template <class IO>
__host__ __device__ constexpr int scan_loaders() { return in_parts<IO>() == 1 ? 2 : 4; }

// One scan workgroup: W tiles of 16 value columns of one head, each computed by a team of T waves
// that share out the state's r axis, and NL waves that load.
//
// The chain of products from one chunk's state to the next bounds the scan, not their number: a
// team shortens it.  Each of its waves keeps r / T of the state, multiplies that part of K and Q,
// and the team adds the parts of K H^T through LDS, in the same order in every wave, so that all
// of them continue with the same R, E and U.
//
// The loading waves bring what a chunk needs into LDS without passing registers, a chunk ahead,
// into the buffer that its predecessor has just left: the phases of a chunk are ordered so that
// between the last read of a buffer and the first read of its next contents lies another phase's
// matrix work.  They count their own loads; the computing waves meet them at barriers only.
// (Computing waves that issued the loads themselves: bf16, 160 heads, 291 against 232 us; loads
// into registers there: 1084 us.)
//
// Measured with outputs, p = 64, r = 128, a chunk in each launch shape: bf16 4.1 us (four single
// waves, 160 workgroups on as many CUs, so that 96 of the 256 stand idle: 64 chunks 260 us; 3.6 and
// 232 with y's operands in two parts, whose y misses the nearest bf16 value once in 400); fp32
// 3.4 us (one team), 6.1 us (two teams), 9.7 us (four waves).  Single waves in fp32 at 256 tiles: 4.9 ms
// for 1024 chunks against 3.5 ms by teams.  A team's sums cost more than its shorter chain wins where
// the chip is full of single waves.
//
// fp32 keys and queries are cut into parts by the loading waves: written as parts by the
// preparation they are half as large again in every read (32 heads of 1024 chunks: preparation 1314,
// scan 1175 us, against 683 and 1238); four loading waves beside the computing ones cost a scan that is
// bound by the vector unit something (96 heads of 32 chunks: 165 -> 197 us, preparation 121 -> 82).
//
// Where few heads leave most of the chip idle, the forward's chunks are cut into segments that run
// side by side.  A segment maps its entry state by rows: h -> h T + b, the same T [r, r] for every
// row.  kCarry runs the recurrence through each segment but the last, on p more rows than r: the
// value columns from zero, which gives b, and r columns with v = 0 from the rows of the identity,
// which gives T (of the first segment only the value columns, from init).  k_delta_join then
// goes from segment to segment, and the outputs start from what it leaves.
template <class IO, int R, int W, int TM, ScanMode MODE>
struct Scan {
    using T = typename IO::T;
    static constexpr int NP = in_parts<IO>(), RP = R < 32 ? 32 : R, KJ = RP / 32;
    static constexpr int JW = KJ / TM, RT = RP / 16 / TM;  // steps of r and state tiles of one wave
    static constexpr bool CUT = through_registers<IO, R>();
    static constexpr int PK = p_kilobytes<IO>(MODE == kReverse);
    static constexpr int QT = 4 * KJ;  // tiles per part
    static constexpr int NL = scan_loaders<IO>(), CW = W * TM;
    static constexpr int TT = 4 / TM;  // token tiles that a wave finishes for its team
    // LDS, bytes
    static constexpr bool LEAN = MODE == kRecord || MODE == kCarry;  // neither q nor P
    static constexpr int KBYTES = NP * QT * 1024, KBUFS = LEAN ? 2 : 1;
    static constexpr int QBYTES = LEAN ? 0 : KBYTES;
    static constexpr int MBYTES = 3 * DTRI * 1024, PBYTES = LEAN ? 0 : PK * DTRI * 1024;
    static constexpr int VBYTES = DL * 16 * W * sizeof(T);
    static constexpr int oK = 0, oQ = oK + KBUFS * KBYTES, oM = oQ + QBYTES, oP = oM + MBYTES, oV = oP + PBYTES,
                         oC = oV + VBYTES, oX = oC + 2 * 4 * DCF, LDS = oX + (TM > 1 ? CW * 4096 : 0);
    // loads of one loading wave
    static constexpr int per(int n) { return (n + NL - 1) / NL; }
    static constexpr int nK = CUT ? 0 : per(QT), nQ = nK, nM = per(3 * DTRI), nP = per(PK * DTRI),
                         nV = per(VBYTES / 1024), nC = 1;

    char* sm;
    const DeltaShape& d;
    const DeltaScan<T>& a;
    int lane, w, tm, i, g, pt, p0, pw, h, b, hk, chunks, len;
    int seg, c0, c1;  // the segment and its chunks
    int64_t bh;

    __device__ Scan(char* smem, const DeltaShape& dd, const DeltaScan<T>& aa, int64_t blk) : sm(smem), d(dd), a(aa) {
        lane = threadIdx.x & 63;
        w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        i = lane & 15;
        g = lane >> 4;
        pt = w / TM;  // tile of the workgroup
        tm = w % TM;  // place in its team
        const int pbs = d.P / (16 * W);
        seg = 0;
        if constexpr (MODE == kCarry) {
            const int all = pbs + d.R / (16 * W), per = pbs + (a.segs - 2) * all;
            int at = static_cast<int>(blk % per);
            bh = blk / per;
            if (at >= pbs) {
                seg = 1 + (at - pbs) / all;
                at = (at - pbs) % all;
            }
            pw = at * 16 * W;
        } else {
            pw = static_cast<int>(blk % pbs) * 16 * W;  // the workgroup's first column
            bh = blk / pbs;
            if constexpr (MODE == kOutputs) {
                seg = static_cast<int>(bh % a.segs);
                bh /= a.segs;
            }
        }
        p0 = pw + 16 * pt;  // the team's
        h = static_cast<int>(bh % d.H);
        b = static_cast<int>(bh / d.H);
        hk = h / (d.H / d.HK);
        len = a.len ? static_cast<int>(a.len[b]) : d.S;
        chunks = (len + DL - 1) / DL;
        c0 = 0;
        c1 = chunks;
        if constexpr (MODE == kOutputs || MODE == kCarry) {
            c0 = seg * a.seg_chunks;
            if (c0 > chunks) c0 = chunks;
            if (c1 > c0 + a.seg_chunks) c1 = c0 + a.seg_chunks;
        }
    }

    // -------------------------------------------------------------- loads into LDS
    __device__ int unit(int m, int n) const {  // this loading wave's m-th of n: each loads as often
        const int t = w - CW + m * NL;
        return n % NL == 0 || t < n ? t : n - 1;
    }
    template <int N>  // N kilobytes, as they are
    __device__ void copy_tiles(int at, const uint16_t* src) const {
        const uint32_t dst = lds_addr(sm) + at;
#pragma unroll
        for (int m = 0; m < per(N); ++m) load_to_lds(src + unit(m, N) * DTILE + lane * 8, dst + unit(m, N) * 1024);
    }
    // Tokens of chunk c of q or k.  Rows past the length repeat its last row: what they feed is
    // multiplied by the zeros of beta and e^G there.  f(this wave's m-th tile, the tile, the address).
    template <class F>
    __device__ void each_qk(const T* x, const int64_t (&stride)[3], int c, F&& f) const {
        const int gs = lane >> 4, is = (lane & 15) ^ (4 * gs);
        const int last = (len - c * DL < DL ? len - c * DL : DL) - 1;
        const T* base = x + b * stride[0] + static_cast<int64_t>(c) * DL * stride[1] + hk * stride[2] +
                        (8 * gs < R ? 8 * gs : 0);
#pragma unroll
        for (int m = 0; m < QT / NL; ++m) {
            const int tile = w - CW + m * NL, tau = tile / KJ, j = tile % KJ, row = 16 * tau + is;
            f(m, tile, base + (row < last ? row : last) * stride[1] + 32 * j);
        }
    }
    __device__ void load_qk(int at, const T* x, const int64_t (&stride)[3], int c) const {
        const uint32_t dst = lds_addr(sm) + at;
        each_qk(x, stride, c, [&](int, int tile, const T* src) { load_to_lds(src, dst + tile * 1024); });
    }
    // The same through registers: fetched a chunk ahead, cut and written when the buffer is free.
    typedef T raw8 __attribute__((ext_vector_type(8)));
    typedef raw8 Ahead[QT / NL];
    __device__ void fetch_qk(Ahead& r, const T* x, const int64_t (&stride)[3], int c) const {
        each_qk(x, stride, c, [&](int m, int, const T* src) { r[m] = *reinterpret_cast<const raw8*>(src); });
    }
    __device__ void put_qk(int at, const Ahead& r) const {
#pragma unroll
        for (int m = 0; m < QT / NL; ++m) {
            const auto x = parts_of<IO>(r[m], R >= 32 || lane < 2 * R);  // 16 lanes for 8 columns
#pragma unroll
            for (int n = 0; n < NP; ++n)
                *reinterpret_cast<b8v*>(sm + at + (n * QT + w - CW + m * NL) * 1024 + lane * 16) = x.p[n];
        }
    }
    // Tokens of chunk c of v or dy, the workgroup's columns, row-major.
    __device__ void load_v(const T* x, int64_t sb, int64_t st, int64_t sh, int c) const {
        constexpr int U = 16 * W * sizeof(T) / 16;  // 16-byte units of a row
        const int last = (len - c * DL < DL ? len - c * DL : DL) - 1;
        const T* base = x + b * sb + static_cast<int64_t>(c) * DL * st + h * sh + (MODE == kCarry && pw >= d.P ? 0 : pw);
#pragma unroll
        for (int m = 0; m < nV; ++m) {
            const int n = unit(m, VBYTES / 1024), u = n * 64 + lane, row = u / U;
            load_to_lds(base + (row < last ? row : last) * st + (u % U) * (16 / static_cast<int>(sizeof(T))),
                        lds_addr(sm) + oV + n * 1024);
        }
    }
    __device__ void load_coef(int c, int buf) const {
        load_to_lds(a.coef + (bh * d.N + c) * DCOEF + 4 * lane, lds_addr(sm) + oC + (buf & 1) * 4 * DCF);
    }

    // -------------------------------------------------------------- operands
    // j, rho: of this wave's share of r
    __device__ Parts<NP> row_op(int base, int tau, int j) const {  // rows: tokens 16 tau + i
        Parts<NP> o;
#pragma unroll
        for (int n = 0; n < NP; ++n)
            o.p[n] = *reinterpret_cast<const b8v*>(sm + base + (n * QT + tau * KJ + tm * JW + j) * 1024 +
                                                    tile_slot(i, g) * 16);
        return o;
    }
    // Rows r = 32 (rho / 2) + 8 (i / 4) + 4 (rho % 2) + i % 4 of the transposed matrix, k over the
    // tokens 32 j + {4 g + v, 16 + 4 g + v}.  Row 4 g + v of state tile rho is then
    // r = 32 (rho / 2) + 8 g + 4 (rho % 2) + v: two state tiles hold eight consecutive r per lane.
    __device__ Parts<NP> col_op(int base, int rho, int j) const {
        Parts<NP> o;
        const int at = base + (2 * j * KJ + tm * JW + (rho >> 1)) * 1024 + tile_slot(4 * g + (i >> 2), i & 3) * 16 +
                       (rho & 1) * 8;
#pragma unroll
        for (int n = 0; n < NP; ++n)
            o.p[n] = join8(lds_col4(reinterpret_cast<const uint16_t*>(sm + at + n * QT * 1024)),
                           lds_col4(reinterpret_cast<const uint16_t*>(sm + at + (n * QT + KJ) * 1024)));
        return o;
    }
    template <int N>
    __device__ Parts<N> tri_op(int base, int tile) const {
        Parts<N> o;
#pragma unroll
        for (int n = 0; n < N; ++n)
            o.p[n] = *reinterpret_cast<const b8v*>(sm + base + (n * DTRI + tile) * 1024 + lane * 16);
        return o;
    }
    __device__ b8v tri_part(int base, int n, int tile) const {
        return *reinterpret_cast<const b8v*>(sm + base + (n * DTRI + tile) * 1024 + lane * 16);
    }
    // v or dy in result layout: tokens 16 t + 4 g + v of value column p0 + i
    __device__ v4f value(int t) const {
        if constexpr (sizeof(T) == 2) {
            const s4 x = lds_col4(reinterpret_cast<const uint16_t*>(sm + oV) + (16 * t + 4 * g + (i >> 2)) * (16 * W) +
                                  16 * pt + 4 * (i & 3));
            return v4f{bf16_to_f32(x[0]), bf16_to_f32(x[1]), bf16_to_f32(x[2]), bf16_to_f32(x[3])};
        } else {
            const float* x = reinterpret_cast<const float*>(sm + oV) + (16 * t + 4 * g) * (16 * W) + 16 * pt + i;
            return v4f{x[0], x[16 * W], x[32 * W], x[48 * W]};
        }
    }
    __device__ const float* coef(int c) const { return reinterpret_cast<const float*>(sm + oC + (c & 1) * 4 * DCF); }
    __device__ static v4f at4(const float* p) { return *reinterpret_cast<const v4f*>(p); }

    // -------------------------------------------------------------- states
    __device__ int row_of(int rho) const { return 32 * (tm * JW + (rho >> 1)) + 8 * g + 4 * (rho & 1); }
    // This lane's row (value column p0 + i) of a state [rows, r], or null.
    __device__ const float* state_row(const float* src, int64_t at, int rows) const {
        return src ? src + (at * rows + p0 + i) * R : nullptr;
    }
    __device__ float* carry_row(int of) const {  // what segment `of` leaves
        return const_cast<float*>(state_row(a.carry, bh * (a.segs - 1) + of, d.P + R));
    }
    __device__ void load_state(v4f (&s)[RT], const float* row) const {
#pragma unroll
        for (int rho = 0; rho < RT; ++rho) {
            const int r = row_of(rho);
            s[rho] = row && r < R ? at4(row + r) : zero4();
        }
    }
    __device__ void unit_state(v4f (&s)[RT]) const {
#pragma unroll
        for (int rho = 0; rho < RT; ++rho)
#pragma unroll
            for (int v = 0; v < 4; ++v) s[rho][v] = row_of(rho) + v == p0 - d.P + i ? 1.0f : 0.0f;
    }
    __device__ void store_state(const v4f (&s)[RT], float* row) const {
#pragma unroll
        for (int rho = 0; rho < RT; ++rho) {
            const int r = row_of(rho);
            if (row && r < R) *reinterpret_cast<v4f*>(row + r) = s[rho];
        }
    }
    // A chunk's state for the gradient kernel, [r, P] rows.
    __device__ void record_state(const v4f (&s)[RT], float* dst, int c) const {
        float* o = dst + (bh * d.N + c) * (static_cast<int64_t>(R) * d.P) + p0 + i;
#pragma unroll
        for (int rho = 0; rho < RT; ++rho) {
            const int r = row_of(rho);
            if (r < R) {
#pragma unroll
                for (int v = 0; v < 4; ++v) o[(r + v) * d.P] = s[rho][v];
            }
        }
    }
    __device__ v4f own(const v4f (&x)[4], int t) const {  // x[tm TT + t]
        v4f o = x[t];
#pragma unroll
        for (int m = 1; m < TM; ++m)
#pragma unroll
            for (int v = 0; v < 4; ++v) o[v] = tm == m ? x[m * TT + t][v] : o[v];
        return o;
    }
    __device__ void record_rows(const v4f (&x)[4], float* dst, int c) const {  // this wave's token tiles
        float* o = dst + ((bh * d.N + c) * DL + 16 * tm * TT) * static_cast<int64_t>(d.P) + p0 + i;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const v4f r = own(x, t);
#pragma unroll
            for (int v = 0; v < 4; ++v) o[(16 * t + 4 * g + v) * d.P] = r[v];
        }
    }
    // c <- c + X s^T (SWAP: its transpose) over this wave's share of r, X = k or q in LDS, from the
    // state's parts, or parts made on the way (MAKE): a step's operands are read, and the next
    // step's parts made, while the matrix cores are at the step before.
    template <bool SWAP, bool MAKE>
    __device__ void rows_product(v4f (&c)[4], int base, Parts<3> (&sp)[JW], const v4f (&s)[RT]) const {
        Parts<NP> op[2][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) op[0][t] = row_op(base, t, 0);
        if constexpr (MAKE) sp[0] = split44<3>(s[0], s[1]);
#pragma unroll
        for (int j = 0; j < JW; ++j) {
            if (j + 1 < JW) {
#pragma unroll
                for (int t = 0; t < 4; ++t) op[(j + 1) & 1][t] = row_op(base, t, j + 1);
            }
            fence();
            if constexpr (SWAP)
                mma_b(c, sp[j], op[j & 1]);
            else
                mma_a(c, op[j & 1], sp[j]);
            if (MAKE && j + 1 < JW) {
                sp[j + 1] = split44<3>(s[2 * j + 2], s[2 * j + 3]);
                mix<4 * terms(NP, 3), 176 / (4 * terms(NP, 3)) / 4 + 1>();
            }
            fence();
        }
    }
    static constexpr int terms(int na, int nb) {
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
    // s <- s + X^T z over the chunk's tokens, X = k or q in LDS, z in result layout
    static constexpr int G = RT < 4 ? RT : 4;  // state tiles at a time
    __device__ void col_ops(Parts<NP> (&op)[G], int base, int step) const {  // step: j, then tiles
#pragma unroll
        for (int m = 0; m < G; ++m) op[m] = col_op(base, step % (RT / G) * G + m, step / (RT / G));
    }
    __device__ void add_outer(v4f (&s)[RT], int base, const v4f (&z)[4]) const {
        constexpr int STEPS = 2 * (RT / G);
        Parts<NP> op[2][G];
        col_ops(op[0], base, 0);
        Parts<3> zp[2];
        zp[0] = split44<3>(z[0], z[1]);
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            if (k + 1 < STEPS) col_ops(op[(k + 1) & 1], base, k + 1);
            fence();
            mma_a(*reinterpret_cast<v4f(*)[G]>(&s[k % (RT / G) * G]), op[k & 1], zp[k / (RT / G)]);
            if (k == 0) {
                zp[1] = split44<3>(z[2], z[3]);
                mix<G * terms(NP, 3), 48 / (G * terms(NP, 3)) + 1>();
            }
            fence();
        }
    }
    // c <- c + A x for a triangular operand in LDS, x in result layout
    template <bool LOWER>
    __device__ void tri_product(v4f (&c)[4], int base, const v4f (&x)[4]) const {
        constexpr int jf = LOWER ? 0 : 1, js = 1 - jf, t0 = LOWER ? 2 : 0;  // the full step, the half one
        Parts<3> a4[4], a2[2];
#pragma unroll
        for (int t = 0; t < 4; ++t) a4[t] = tri_op<3>(base, LOWER ? tri_lower(t, jf) : tri_upper(t, jf));
        const auto x0 = split44<3>(x[2 * jf], x[2 * jf + 1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) a2[t] = tri_op<3>(base, LOWER ? tri_lower(t0 + t, js) : tri_upper(t0 + t, js));
        fence();
        mma_a(c, a4, x0);
        const auto x1 = split44<3>(x[2 * js], x[2 * js + 1]);
        mix<16, 3>();
        fence();
        mma_a(*reinterpret_cast<v4f(*)[2]>(&c[t0]), a2, x1);
    }

    // -------------------------------------------------------------- a team's sums
    __device__ v4f* share(int member, int t) const {
        return reinterpret_cast<v4f*>(sm + oX + (pt * TM + member) * 4096 + t * 1024) + lane;
    }
    __device__ void team_sum(v4f (&x)[4]) const {  // the sum of the members' x, in all of them
        if constexpr (TM > 1) {
#pragma unroll
            for (int t = 0; t < 4; ++t) *share(tm, t) = x[t];
            meet();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                x[t] = *share(0, t);
#pragma unroll
                for (int m = 1; m < TM; ++m) x[t] += *share(m, t);
            }
        }
    }

    // An operand tile of P as it lies in LDS, and its parts.
    struct PTile {
        v4f x[PK];
    };
    __device__ PTile p_tile(int tile) const {
        PTile o;
#pragma unroll
        for (int n = 0; n < PK; ++n)
            o.x[n] = at4(reinterpret_cast<const float*>(sm + oP + (n * DTRI + tile) * 1024 + lane * 16));
        return o;
    }
    __device__ static Parts<3> p_parts(const PTile& p) {
        if constexpr (PK == 2)
            return split44<3>(p.x[0], p.x[1]);
        else
            return __builtin_bit_cast(Parts<3>, p);
    }
    // y <- y + P u for this wave's token tiles; what is left to cut for the second step is cut while
    // the matrix cores are at the first
    __device__ void intra(v4f (&y)[TT], const v4f (&u)[4]) const {
        constexpr int T2 = TM == 1 ? 2 : 0;  // the first tile that reaches the second step
        PTile raw[2][TT];
        const bool two = TM == 1 || tm >= TM / 2;
#pragma unroll
        for (int t = 0; t < TT; ++t) raw[0][t] = p_tile(tri_lower(tm * TT + t, 0));
        if (two) {
#pragma unroll
            for (int t = T2; t < TT; ++t) raw[1][t] = p_tile(tri_lower(tm * TT + t, 1));
        }
        Parts<3> op[TT], op1[TT - T2];
#pragma unroll
        for (int t = 0; t < TT; ++t) op[t] = p_parts(raw[0][t]);
        const auto u0 = split44<3>(u[0], u[1]);
        fence();
        mma_b(y, u0, op);
        if (two) {
            const auto u1 = split44<3>(u[2], u[3]);
#pragma unroll
            for (int t = T2; t < TT; ++t) op1[t - T2] = p_parts(raw[1][t]);
            if constexpr (TM == 1) {
                mix<4 * terms(3, 3), PK == 2 ? 7 : 3>();
                fence();
            }
            mma_b(*reinterpret_cast<v4f(*)[TT - T2]>(&y[T2]), u1, op1);
        }
    }

    // -------------------------------------------------------------- the forward recurrence
    __device__ void store_y(const v4f (&y)[TT], int c) const {  // D[p][t]: token 16 t + i, columns 4 g + v
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int64_t tok = static_cast<int64_t>(c) * DL + 16 * (tm * TT + t) + i;
            // past the length zeros as they are: as products they would be NaN beside a NaN or an infinity
            if (tok < d.S)
                io<IO>::st4(a.y, ((b * static_cast<int64_t>(d.S) + tok) * d.H + h) * d.P + p0 + 4 * g,
                            tok < len ? y[t] : zero4());
        }
    }

    // Waits count the loads into LDS that were issued after the ones waited for; those into registers
    // are the compiler's to wait for, and only make these waits end later.
    __device__ void load_forward() const {
        auto m = [&](int c) {
            copy_tiles<3 * DTRI>(oM, a.M + (bh * d.N + c) * (3 * DTRI * DTILE));
            load_v(a.v, d.vs[0], d.vs[1], d.vs[2], c);
        };
        Ahead kr, qr;
        if constexpr (MODE == kOutputs) {
            if constexpr (CUT) {
                fetch_qk(qr, a.q, d.qs, c0);
                fetch_qk(kr, a.k, d.ks, c0);
                put_qk(oQ, qr);
                if (c0 + 1 < c1) fetch_qk(qr, a.q, d.qs, c0 + 1);
            } else {
                load_qk(oQ, a.q, d.qs, c0);
            }
            load_coef(c0, c0);
            m(c0);
            if constexpr (!CUT) load_qk(oK, a.k, d.ks, c0);
            for (int c = c0; c < c1; ++c) {
                const bool more = c + 1 < c1;
                wait_barrier<nM + nV + nK>();  // q and the coefficients
                if constexpr (CUT) put_qk(oK, kr);
                copy_tiles<PK * DTRI>(oP, a.P + (bh * d.N + c) * (PK * DTRI * DTILE));
                wait_barrier<nP>();  // M, v and k
                if (more) {
                    if constexpr (CUT)
                        put_qk(oQ, qr);
                    else
                        load_qk(oQ, a.q, d.qs, c + 1);
                    load_coef(c + 1, c + 1);
                    if constexpr (CUT) fetch_qk(kr, a.k, d.ks, c + 1);
                }
                if constexpr (TM > 1) wait_barrier<63>();
                wait_barrier<63>();
                if (more) {
                    m(c + 1);
                    wait_barrier<nQ + nC + nM + nV>();  // P
                    if constexpr (!CUT)
                        load_qk(oK, a.k, d.ks, c + 1);
                    else if (c + 2 < c1)
                        fetch_qk(qr, a.q, d.qs, c + 2);
                } else {
                    wait_barrier<0>();
                }
            }
        } else {
            auto buf = [](int c) { return oK + (c & 1) * KBYTES; };
            if constexpr (CUT) {
                fetch_qk(kr, a.k, d.ks, c0);
                put_qk(buf(c0), kr);
                if (c0 + 1 < c1) fetch_qk(kr, a.k, d.ks, c0 + 1);
            } else {
                load_qk(buf(c0), a.k, d.ks, c0);
            }
            load_coef(c0, c0);
            m(c0);
            for (int c = c0; c < c1; ++c) {
                const bool more = c + 1 < c1;
                wait_barrier<0>();
                if (more) {
                    if constexpr (CUT) {
                        put_qk(buf(c + 1), kr);
                        if (c + 2 < c1) fetch_qk(kr, a.k, d.ks, c + 2);
                    } else {
                        load_qk(buf(c + 1), a.k, d.ks, c + 1);
                    }
                }
                if constexpr (TM > 1) wait_barrier<63>();
                wait_barrier<63>();
                if (more) {
                    m(c + 1);
                    load_coef(c + 1, c + 1);
                }
            }
        }
    }

    __device__ void forward() const {
        // a segment after which the row ends (or that starts past its end) need not be carried
        if (MODE == kCarry && c0 + a.seg_chunks >= chunks) return;
        if (w >= CW) {
            if (c0 < c1) load_forward();
            return;
        }
        const bool values = MODE != kCarry || p0 < d.P;
        v4f s[RT];
        if (!values)
            unit_state(s);
        else if (seg == 0)
            load_state(s, state_row(a.init, bh, d.P));
        else
            load_state(s, MODE == kOutputs && c0 < c1 ? carry_row(seg - 1) : nullptr);
        int c = c0;
        for (; c < c1; ++c) {
            const int kb = oK + (LEAN ? (c & 1) * KBYTES : 0);
            v4f x[4], y[4], u[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = y[t] = u[t] = zero4();
            Parts<3> sp[JW];
            meet();  // outputs: q and the coefficients are here, P is free; else everything is here
            const float* cf = coef(c);
            if constexpr (MODE == kOutputs) {
                rows_product<true, true>(y, oQ, sp, s);
                meet();  // M, v and k are here, q is free
                rows_product<false, false>(x, kb, sp, s);
            } else {
                rows_product<false, true>(x, kb, sp, s);
            }
            team_sum(x);
            // R = v - e^G x, E = M R (value column p0 + i, tokens 16 t + 4 g + v)
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = (values ? value(t) : zero4()) - at4(cf + 16 * t + 4 * g) * x[t];
            tri_product<true>(u, oM, x);
            v4f z[4];
            meet();  // M and v are free
            if constexpr (MODE == kRecord) {
                record_state(s, a.H, c);
                record_rows(u, a.E, c);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u[t] *= at4(cf + 2 * DL + 16 * t + 4 * g);
                z[t] = u[t] * at4(cf + DL + 16 * t + 4 * g);
            }
            const float eL = cf[3 * DL];
#pragma unroll
            for (int r = 0; r < RT; ++r) s[r] *= eL;
            if constexpr (MODE == kOutputs && TM > 1) {
#pragma unroll
                for (int t = 0; t < 4; ++t) *share(tm, t) = y[t];
            }
            add_outer(s, kb, z);
            if constexpr (MODE == kOutputs) {
                meet();  // P is here, k is free, the team's parts of q H are written
                v4f yo[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if constexpr (TM == 1) {
                        yo[t] = y[t];
                    } else {
                        yo[t] = *share(0, tm * TT + t);
#pragma unroll
                        for (int m = 1; m < TM; ++m) yo[t] += *share(m, tm * TT + t);
                    }
                    yo[t] *= d.scale * cf[16 * (tm * TT + t) + i];
                }
                intra(yo, u);
                store_y(yo, c);
            }
            mfma_settle();
        }
        if constexpr (MODE == kCarry) store_state(s, carry_row(seg));
        if constexpr (MODE == kOutputs) {
            // the segment that holds the row's last chunk, or the first one of an empty row
            if (c1 == chunks && (c0 < c1 || seg == 0)) store_state(s, const_cast<float*>(state_row(a.final_state, bh, d.P)));
            v4f zero[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) zero[t] = zero4();
            const int end = (seg + 1) * a.seg_chunks < d.N ? (seg + 1) * a.seg_chunks : d.N;
            if (c < seg * a.seg_chunks) c = seg * a.seg_chunks;
            for (; c < end; ++c) store_y(zero, c);  // chunks past the row's length
        }
    }

    // u <- u + P^T dy for step j of this wave's token tiles
    __device__ void intra_t(v4f (&u)[TT], const Parts<NP>& y, int j) const {
#pragma unroll
        for (int s0 = 2; s0 >= 0; --s0)
#pragma unroll
            for (int n = 0; n <= s0; ++n)
                if (s0 - n < NP)
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        if (TM == 1 && j < t / 2) continue;
                        const int tile = tri_upper(tm * TT + t, j);
                        u[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(tri_part(oP, n, tile), y.p[s0 - n], u[t], 0, 0, 0);
                    }
    }

    // -------------------------------------------------------------- the reverse recurrence
    __device__ void load_reverse() const {
        const int64_t tok = static_cast<int64_t>(d.H) * d.P;
        auto front = [&](int c) {  // what the first two phases read
            copy_tiles<3 * DTRI>(oP, a.P + (bh * d.N + c) * (3 * DTRI * DTILE));
            if constexpr (!CUT) load_qk(oQ, a.q, d.qs, c);
            load_v(a.dy, d.S * tok, tok, d.P, c);
            load_coef(c, c);
        };
        const int last = chunks - 1;
        Ahead kr, qr;
        if constexpr (CUT) {
            fetch_qk(qr, a.q, d.qs, last);
            fetch_qk(kr, a.k, d.ks, last);
            put_qk(oQ, qr);
            if (last > 0) fetch_qk(qr, a.q, d.qs, last - 1);
        }
        front(last);
        copy_tiles<3 * DTRI>(oM, a.NT + (bh * d.N + last) * (3 * DTRI * DTILE));
        if constexpr (!CUT) load_qk(oK, a.k, d.ks, last);
        for (int c = last; c >= 0; --c) {
            wait_barrier<nM + nK>();  // P^T, q, dy and the coefficients
            if constexpr (CUT) put_qk(oK, kr);
            wait_barrier<0>();  // N^T and k
            if (c > 0) {
                if constexpr (CUT) put_qk(oQ, qr);
                front(c - 1);
                if constexpr (CUT) fetch_qk(kr, a.k, d.ks, c - 1);
            }
            if constexpr (TM > 1) wait_barrier<63>();
            wait_barrier<63>();
            if (c > 0) copy_tiles<3 * DTRI>(oM, a.NT + (bh * d.N + c - 1) * (3 * DTRI * DTILE));
            wait_barrier<63>();
            if constexpr (!CUT) {
                if (c > 0) load_qk(oK, a.k, d.ks, c - 1);
            } else if (c > 1) {
                fetch_qk(qr, a.q, d.qs, c - 2);
            }
        }
    }

    __device__ void reverse() const {
        if (w >= CW) {
            if (chunks > 0) load_reverse();
            return;
        }
        v4f s[RT];
        load_state(s, state_row(a.d_final, bh, d.P));
        for (int c = chunks - 1; c >= 0; --c) {
            v4f u[4], dy[4], x[4], gq[RT];
            meet();  // P^T, q, dy and the coefficients are here
            const float* cf = coef(c);
            record_state(s, a.dH, c);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                dy[t] = value(t);
                x[t] = zero4();
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) gq[r] = zero4();
            // dU = P^T dy + tail (K dH^T): of the first term, this wave's token tiles
            v4f pu[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) pu[t] = zero4();
            if (TM == 1 || tm < (TM + 1) / 2) intra_t(pu, split44<NP>(dy[0], dy[1]), 0);
            intra_t(pu, split44<NP>(dy[2], dy[3]), 1);
#pragma unroll
            for (int t = 0; t < 4; ++t) dy[t] *= d.scale * at4(cf + 16 * t + 4 * g);
            add_outer(gq, oQ, dy);
            meet();  // N^T and k are here, P^T, q and dy are free
            Parts<3> sp[JW];
            rows_product<false, true>(x, oK, sp, s);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u[t] = at4(cf + DL + 16 * t + 4 * g) * x[t];
                if (TM == 1) {
                    u[t] += pu[t % TT];
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v) u[t][v] += t / TT == tm ? pu[t % TT][v] : 0.0f;
                }
                x[t] = zero4();
            }
            team_sum(u);
            tri_product<false>(x, oM, u);
            meet();  // N^T is free
            record_rows(x, a.dZ, c);
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] *= -at4(cf + 16 * t + 4 * g) * at4(cf + 2 * DL + 16 * t + 4 * g);
            const float eL = cf[3 * DL];
#pragma unroll
            for (int r = 0; r < RT; ++r) s[r] = eL * s[r] + gq[r];
            add_outer(s, oK, x);
            meet();  // k is free
            mfma_settle();
        }
        store_state(s, const_cast<float*>(state_row(a.d_init, bh, d.P)));
    }

    // A computing wave's side of a barrier: its LDS reads have returned.
    __device__ static void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
};

}  // namespace

template <class IO, int R, int W, int TM>
__global__ __launch_bounds__(64 * (W * TM + scan_loaders<IO>()), 2) void k_delta_scan(DeltaShape d,
                                                                                   DeltaScan<typename IO::T> a) {
    using S = Scan<IO, R, W, TM, kOutputs>;
    __shared__ __align__(16) char sm[S::LDS];
    S(sm, d, a, xcd_order(blockIdx.x, gridDim.x)).forward();
}

template <class IO, int R, int W, int TM>
__global__ __launch_bounds__(64 * (W * TM + scan_loaders<IO>()), 2) void k_delta_carry(DeltaShape d,
                                                                                    DeltaScan<typename IO::T> a) {
    using S = Scan<IO, R, W, TM, kCarry>;
    __shared__ __align__(16) char sm[S::LDS];
    S(sm, d, a, xcd_order(blockIdx.x, gridDim.x)).forward();
}

// From segment to segment, per (b, h) and 16 value columns: the state at the end of segment s,
// H_s = H_{s-1} T_s + b_s, in the place of b_s.  Four waves share out the columns of r; the
// products are fp32 MFMAs.
template <int R>
__global__ __launch_bounds__(256) void k_delta_join(DeltaShape d, const int64_t* __restrict__ len, float* carry,
                                                    int segs, int seg_chunks) {
    constexpr int LH = R + 4, RT = (R / 16 + 3) / 4;
    __shared__ __align__(16) float sH[2][16 * LH];
    const int tiles = d.P / 16;
    const int64_t bh = blockIdx.x / tiles;
    const int p0 = 16 * static_cast<int>(blockIdx.x % tiles);
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    const int n = len ? static_cast<int>(len[bh / d.H]) : d.S, chunks = (n + DL - 1) / DL;
    float* of = carry + bh * (segs - 1) * static_cast<int64_t>(d.P + R) * R;
    if (2 * seg_chunks >= chunks) return;  // nothing is carried past the first segment
    for (int x = threadIdx.x; x < 16 * R; x += 256) sH[0][x / R * LH + x % R] = of[p0 * R + x];
    for (int s = 1; (s + 1) * seg_chunks < chunks; ++s) {
        of += static_cast<int64_t>(d.P + R) * R;
        const float *H = sH[(s + 1) & 1], *T = of + d.P * R;
        float *to = sH[s & 1], *b = of + p0 * R;
        v4f acc[RT];
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            const int col = 16 * (w * RT + m) + i;
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[m][v] = col < R ? b[(4 * g + v) * R + col] : 0.0f;
        }
        __syncthreads();
        if (w * RT * 16 < R) {
#pragma unroll
            for (int k = 0; k < R; k += 4)
#pragma unroll
                for (int m = 0; m < RT; ++m)
                    acc[m] = mfma16(H[i * LH + k + g], T[(k + g) * R + 16 * (w * RT + m) + i], acc[m]);
#pragma unroll
            for (int m = 0; m < RT; ++m) {
                const int col = 16 * (w * RT + m) + i;
#pragma unroll
                for (int v = 0; v < 4; ++v) b[(4 * g + v) * R + col] = to[(4 * g + v) * LH + col] = acc[m][v];
            }
        }
    }
}

// Both recurrences of the backward: the first half of the workgroups run the reverse, which takes
// about twice as long, the second half recompute the entry states and E.  Started last, the short
// ones fill in where the chip does not hold all of them at once (bf16, 160 heads of 64 chunks: 630
// us, the other way round 923).  Writes H, dH, E and dZ, 1.17 GB there, at 4.0 TB/s of all traffic.
template <class IO, int R, int W, int TM>
__global__ __launch_bounds__(64 * (W * TM + scan_loaders<IO>()), 2) void k_delta_states(DeltaShape d,
                                                                                     DeltaScan<typename IO::T> a) {
    using F = Scan<IO, R, W, TM, kRecord>;
    using B = Scan<IO, R, W, TM, kReverse>;
    __shared__ __align__(16) char sm[F::LDS > B::LDS ? F::LDS : B::LDS];
    const int64_t half = gridDim.x / 2;
    if (blockIdx.x < half)
        B(sm, d, a, xcd_order(blockIdx.x, half)).reverse();
    else
        F(sm, d, a, xcd_order(blockIdx.x - half, half)).forward();
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
    a.carry = f.carry;
    a.segs = 1;
    a.seg_chunks = 0;
    return a;
}

template <class IO, int R>
hipError_t prep_r(const DeltaShape& d, const DeltaBufs& f, bool bwd, hipStream_t st) {
    const auto a = typed<IO>(f);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(d.B) * d.H * d.N));
    if (bwd)
        k_delta_prep<IO, R, true><<<grid, 256, 0, st>>>(d, a.q, a.k, f.g, f.beta, a.len, a.coef, a.M, a.P,
                                                    a.NT);
    else
        k_delta_prep<IO, R, false><<<grid, 256, 0, st>>>(d, a.q, a.k, f.g, f.beta, a.len, a.coef, a.M, a.P,
                                                     nullptr);
    return hipGetLastError();
}

// Workgroups of one segment and one kind of work.
template <class IO, int R, int W, int TM>
hipError_t scan_w(const DeltaShape& d, const DeltaBufs& f, ScanMode mode, int segs, hipStream_t st) {
    constexpr int NTHR = 64 * (W * TM + scan_loaders<IO>());
    auto a = typed<IO>(f);
    a.segs = segs;
    a.seg_chunks = (d.N + segs - 1) / segs;
    const int64_t heads = static_cast<int64_t>(d.B) * d.H;
    const int pbs = d.P / (16 * W), rbs = d.R / (16 * W);
    if (mode == kReverse) {
        k_delta_states<IO, R, W, TM><<<dim3(static_cast<unsigned>(2 * heads * pbs)), NTHR, 0, st>>>(d, a);
    } else if (mode == kOutputs) {
        k_delta_scan<IO, R, W, TM><<<dim3(static_cast<unsigned>(heads * segs * pbs)), NTHR, 0, st>>>(d, a);
    } else if constexpr (R >= 16 * W) {
        const int per = pbs + (segs - 2) * (pbs + rbs);
        k_delta_carry<IO, R, W, TM><<<dim3(static_cast<unsigned>(heads * per)), NTHR, 0, st>>>(d, a);
    } else {
        return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// The fewest columns per workgroup with which the workgroups still find a CU each; in fp32,
// where a chunk is mostly matrix work, two rounds of teams of two also beat one of single waves.
template <class IO, int R>
hipError_t scan_r(const DeltaShape& d, const DeltaBufs& f, ScanMode mode, int segs, hipStream_t st) {
    constexpr int KJ = R < 32 ? 1 : R / 32;
    const int64_t heads = static_cast<int64_t>(d.B) * d.H;
    const int rows = mode == kCarry && d.R < d.P ? d.R : d.P;  // whole workgroups of either kind of column
    const int64_t tiles = mode == kCarry ? heads * (d.P / 16 + (segs - 2) * ((d.P + d.R) / 16))
                                         : heads * segs * (d.P / 16);
    const int64_t all = mode == kReverse ? 2 * tiles : tiles;
    const int W = all <= 256 || rows < 32 ? 1 : (in_parts<IO>() == 3 ? tiles : all) <= 512 || rows < 64 ? 2 : 4;
    const int TM = W <= 2 && KJ >= 2 ? 2 : 1;
    if constexpr (KJ >= 2) switch (10 * W + TM) {
        case 12: return scan_w<IO, R, 1, 2>(d, f, mode, segs, st);
        case 22: return scan_w<IO, R, 2, 2>(d, f, mode, segs, st);
        case 41: return scan_w<IO, R, 4, 1>(d, f, mode, segs, st);
    } else switch (W) {
        case 1: return scan_w<IO, R, 1, 1>(d, f, mode, segs, st);
        case 2: return scan_w<IO, R, 2, 1>(d, f, mode, segs, st);
        case 4: return scan_w<IO, R, 4, 1>(d, f, mode, segs, st);
    }
    return hipErrorInvalidValue;
}

template <class F>
hipError_t by_r(const DeltaShape& d, F&& f) {
    switch (d.R) {
        case 16: return f(std::integral_constant<int, 16>{});
        case 32: return f(std::integral_constant<int, 32>{});
        case 64: return f(std::integral_constant<int, 64>{});
        case 128: return f(std::integral_constant<int, 128>{});
        default: return hipErrorInvalidValue;
    }
}

hipError_t scan(const DeltaShape& d, const DeltaBufs& f, ScanMode mode, int segs, hipStream_t st) {
    return by_r(d, [&](auto r) {
        constexpr int R = decltype(r)::value;
        return d.io == 1 ? scan_r<BF16, R>(d, f, mode, segs, st) : scan_r<F32, R>(d, f, mode, segs, st);
    });
}

}  // namespace

// Microseconds that `tiles` tiles of 16 state rows take for a chunk each (p = 64, r = 128), with
// outputs or only carried: in one round of teams on their own, in one of teams on a CU by twos, or in
// rounds of four tiles a CU (which scan_r goes by); of two, where rows of fewer than 64 leave a
// workgroup no four tiles.
static int64_t chunk_time(const DeltaShape& d, int64_t tiles, bool outputs) {
    static const int us[2][2][3] = {{{4, 4, 5}, {4, 7, 10}}, {{2, 3, 3}, {3, 3, 4}}};
    const int* t = us[d.io][outputs];
    if (tiles <= 256) return t[0];
    if ((outputs || d.P < d.R ? d.P : d.R) < 64) return t[1] * ((tiles + 511) / 512);
    return tiles <= 512 ? t[1] : t[2] * ((tiles + 1023) / 1024);
}

// The number of segments with the shortest way: of a segment the chunks, carried and then with
// outputs, and the joins (6 us each).  A sequence is left whole unless that saves a fifth.  Measured
// on both sides, whole and in 3 to 32 segments, at 552 shapes: both io types, nine (p, r) from 16 to 128,
// 16 to 1024 chunks, 1 to 256 tiles.  None of the 260 that the rule cuts is slower so, and the median takes
// 0.44 of its time (p = 64, r = 128: fp32, 8 heads, 4096 tokens, 290 -> 110 us; 32 heads, 65,536 tokens,
// 5.2 -> 3.0 ms; bf16, 8 heads, 4096 tokens, 188 -> 82 us; 32 heads, 16,384 tokens, 801 -> 504 us).  Those it
// leaves whole would win a twelfth at the median and three quarters at most.  With rounds of four tiles for
// narrow states too, twelve more were cut that run 4 to 25 % longer so (bf16, p = 16, r = 128, 96 heads,
// 16,384 tokens: 1008 -> 1262 us).
int delta_segments(const DeltaShape& d) {
    const int64_t heads = static_cast<int64_t>(d.B) * d.H, p = d.P / 16, r = d.R / 16;
    if (d.N < 16 || heads * p > 256) return 1;  // (few chunks; heads that fill the chip)
    int64_t best = d.N * chunk_time(d, heads * p, true) * 4 / 5;
    int segs = 1;
    for (int n = 3; n <= d.N / 4 && n * heads * p <= 1024; ++n) {
        const int64_t chunks = (d.N + n - 1) / n, carried = heads * (p + (n - 2) * (p + r));
        const int64_t way = chunks * (chunk_time(d, carried, false) + chunk_time(d, n * heads * p, true)) + 6 * n;
        if (way < best) {
            best = way;
            segs = n;
        }
    }
    return segs;
}

hipError_t launch_delta_prep(const DeltaShape& d, const DeltaBufs& f, bool bwd, hipStream_t st) {
    return by_r(d, [&](auto r) {
        constexpr int R = decltype(r)::value;
        return d.io == 1 ? prep_r<BF16, R>(d, f, bwd, st) : prep_r<F32, R>(d, f, bwd, st);
    });
}

hipError_t launch_delta_carry(const DeltaShape& d, const DeltaBufs& f, int segs, hipStream_t st) {
    return scan(d, f, kCarry, segs, st);
}

hipError_t launch_delta_join(const DeltaShape& d, const DeltaBufs& f, int segs, hipStream_t st) {
    return by_r(d, [&](auto r) {
        const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(d.B) * d.H * (d.P / 16)));
        k_delta_join<decltype(r)::value><<<grid, 256, 0, st>>>(d, f.len, f.carry, segs, (d.N + segs - 1) / segs);
        return hipGetLastError();
    });
}

hipError_t launch_delta_scan(const DeltaShape& d, const DeltaBufs& f, int segs, hipStream_t st) {
    return scan(d, f, kOutputs, segs, st);
}

hipError_t launch_delta_states(const DeltaShape& d, const DeltaBufs& f, hipStream_t st) {
    return scan(d, f, kReverse, 1, st);
}

}  // namespace ssd
