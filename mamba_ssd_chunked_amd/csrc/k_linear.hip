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
// dY itself is not made: <dy, dY> = <T, W> + <H, W'> + sum_{s<t} (t-s) P_ts (dy_t.v_s) scale, with
// W = scale sum_t a^{t+1} dy_t q_t^T and W' the same (t+1) times.
//
// Tokens past a row's length are zeros in every operand; their memory is not read.
#include "linear_scan.hpp"

namespace ssd {

// Waves of a SIMD that share its registers: two, but one for the outputs of narrow fp32 heads with wide keys, which
// take 287 (two waves would have 256 each).
template <class IO, int R, int NW, int MODE>
constexpr int kLinearWaves = in_parts<IO>() > 1 && R == 128 && NW == 2 && MODE == kOutputs ? 1 : 2;

// Outputs, or what each segment but the last adds to a state.
template <class IO, int R, int NTILE, int NW, int MODE>
__global__ __launch_bounds__(64 * NW, (kLinearWaves<IO, R, NW, MODE>)) void k_linear(LinearShape d, LinearJobs jobs) {
    using Scan = LinearScan<IO, R, NTILE, NW, MODE>;
    __shared__ __align__(16) char sm[Scan::LDS];
    const int pbs = d.P <= Scan::PC ? 1 : d.P / Scan::PC, per = Scan::OUT ? d.segs : d.segs - 1;
    const int64_t blk = linear_order(blockIdx.x, gridDim.x);
    Scan(sm, d, blockIdx.y ? jobs.job[1] : jobs.job[0], blk / pbs / per, static_cast<int>(blk / pbs % per),
         static_cast<int>(blk % pbs) * Scan::PC)
        .run();
}

// From what each segment adds to a state to the states that the segments start from, in place.
// Layout [bh, seg, (H or H and T), p r]; a thread has four elements.
template <bool TAN>
__global__ __launch_bounds__(256) void k_linear_join(LinearShape d, LinearJobs jobs) {
    const LinearJob& a = jobs.job[blockIdx.y];
    const int64_t size = static_cast<int64_t>(d.P) * d.R, quads = size / 4;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t bh = at / quads, q = at % quads;
    if (bh >= static_cast<int64_t>(d.B) * d.H) return;
    const int h = static_cast<int>(bh % d.H), b = static_cast<int>(bh / d.H);
    const int len = d.len ? static_cast<int>(d.len[b]) : d.S;
    const double l2 = log2_decay(d.log_decay[h]);
    const int64_t tokens = static_cast<int64_t>(d.seg_chunks) * LC;
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

namespace {

template <class IO, int R, int P, int MODE>
hipError_t run_p(const LinearShape& d, const LinearJobs& jobs, hipStream_t st) {
    constexpr int NTILE = MODE == kTangentCarry ? 1 : kLinearTiles<IO, P, R>, NW = P <= 32 ? 2 : 4, PC = 16 * NTILE * NW;
    const int64_t per = MODE == kOutputs ? d.segs : d.segs - 1, pbs = P <= PC ? 1 : P / PC;
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(d.B) * d.H * per * pbs), jobs.n);
    k_linear<IO, R, NTILE, NW, MODE><<<grid, 64 * NW, 0, st>>>(d, jobs);
    return hipGetLastError();
}

template <int MODE>
hipError_t run(const LinearShape& d, const LinearJobs& jobs, hipStream_t st) {
    return by_widths(d.P, d.R, [&](auto p, auto r) {
        constexpr int P = decltype(p)::value < 32 ? 32 : decltype(p)::value, R = decltype(r)::value;
        return d.io == 1 ? run_p<BF16, R, P, MODE>(d, jobs, st) : run_p<F32, R, P, MODE>(d, jobs, st);
    });
}

}  // namespace

namespace {

// A gradient in n segments, in us, as measured with p = 64 and r = 128 on a chip of 512 places (two workgroups
// a CU): a chunk of a workgroup takes 5.3 (bf16 3.0), 7.4 (4.0) with the decay's gradient beside it, less alone
// on its CU; beyond the places a round more and half of one for its uneven end.  A chunk carried takes 2 (1), 6
// (4) with the state's derivative, and the launches between 15 or 25.  Narrower states are taken to need less, to a
// floor, in proportion: at twelve shapes of other widths (16 to 128) the rule was within 7 % of the best of 1 to 16
// segments eight times and 12 to 24 % above it four times (bf16, 64 heads of 4096 tokens, 128 x 128, 384 us for 321).
double gradient_time(const LinearShape& d, bool decay, int n) {
    auto rounds = [](double wgs) { return wgs <= 256.0 ? 0.73 : wgs <= 512.0 ? 1.0 : wgs / 512.0 + 0.5; };
    const bool bf = d.io == 1;
    const double heads = static_cast<double>(d.B) * d.H, left = (d.N + n - 1) / n;
    const double chunk = (decay ? (bf ? 4.0 : 7.4) : (bf ? 3.0 : 5.3)) * (0.25 + (d.P + d.R) / 256.0);
    const double t = left * chunk * rounds(heads * linear_grad_blocks(d, decay) * n);
    if (n == 1) return t;
    const double carried = heads * linear_blocks(d) * (n - 1), wide = left * (0.5 + (d.P + d.R) / 384.0);
    return t + (decay ? 25.0 + wide * (bf ? 4.0 : 6.0) * rounds(carried) : 15.0 + wide * (bf ? 1.0 : 2.0) * rounds(2.0 * carried));
}

}  // namespace

// Forwards, as many segments as give 512 places (two workgroups a CU, as the registers allow; bf16 with r = 128 three,
// which does not show in a fourth segment below) a workgroup each, of at least two chunks.  Whole where heads alone take more than half the places, or where the chunks that a workgroup is
// spared (2 us each in bf16 and 3.5 in fp32 with r = 128, half of that with narrow keys) do not pay for
// carrying (half as long a chunk) and for two more launches.  Measured in 1 to 32 segments: bf16, p = 64,
// r = 128, 160 heads of 4096 tokens 272 us whole, 216 in three, 219 in four, 234 in five; 96 of 1531 105 whole, 67 in
// five; 32 of 8192 525 whole, 101 in sixteen; fp32 8 of 1024 126 whole, 33 in sixteen.
// Backwards, where a head has workgroups of several kinds and the rounds end unevenly, the number of segments
// of four chunks or more with the least gradient_time.  Measured in 1 to 24 segments, p = 64, r = 128, with the
// decay's gradient, fp32: 48 heads of 2048 tokens 329 us whole, 391 in two, 291 in eight; 32 of 16384 2509
// whole, 1489 in four, 1196 in sixteen; 160 of 4096 1513 whole, 1445 in four; without it, bf16: 96 of 2048 192
// whole, 184 in four; 160 of 4096 411 whole, 526 in four.
int linear_segments(const LinearShape& d, bool bwd, bool decay) {
    const int64_t heads = static_cast<int64_t>(d.B) * d.H, wgs = heads * (bwd ? linear_grad_blocks(d, decay) : linear_blocks(d));
    if (wgs == 0) return 1;
    if (bwd) {
        int best = 1;
        double least = gradient_time(d, decay, 1);
        for (int n = 2; n <= d.N / 4 && n * wgs <= 2560; n += 1 + n / 8)  // (few: this runs in every call)
            if (const double t = gradient_time(d, decay, n); t < least) best = n, least = t;
        return best;
    }
    if (wgs > 256) return 1;
    int64_t n = 512 / wgs;
    if (n > d.N / 2) n = d.N / 2;
    if (n < 2) return 1;
    const double chunk = (d.io == 1 ? 1.0 : 1.75) * (1.0 + d.R / 128.0), left = static_cast<double>((d.N + n - 1) / n);
    return chunk * d.N < 1.5 * chunk * left + 15.0 ? 1 : static_cast<int>(n);
}
int linear_blocks(const LinearShape& d) { return d.P == 128 && linear_tiles(d.io == 1, d.P, d.R) == 1 ? 2 : 1; }

hipError_t launch_linear_scan(const LinearShape& d, const LinearJobs& jobs, hipStream_t st) {
    return run<kOutputs>(d, jobs, st);
}
hipError_t launch_linear_carry(const LinearShape& d, const LinearJobs& jobs, bool tangent, hipStream_t st) {
    return tangent ? run<kTangentCarry>(d, jobs, st) : run<kCarry>(d, jobs, st);
}
hipError_t launch_linear_join(const LinearShape& d, const LinearJobs& jobs, bool tangent, hipStream_t st) {
    const int64_t quads = static_cast<int64_t>(d.B) * d.H * d.P * d.R / 4;
    const dim3 grid(static_cast<unsigned>((quads + 255) / 256), jobs.n);
    if (tangent)
        k_linear_join<true><<<grid, 256, 0, st>>>(d, jobs);
    else
        k_linear_join<false><<<grid, 256, 0, st>>>(d, jobs);
    return hipGetLastError();
}

}  // namespace ssd
