// Linear attention: the gradients (k_linear.hip states the mathematics).
//
// d_q, d_k and d_v are three scans that need nothing of each other, and so is the derivative along the
// decay: all in one launch, those of a head side by side, so that what two of them read meets in an L2.
// (One launch each, 160 heads of 4096 tokens: d_v 275 us on 160 of the 256 CUs, d_q and d_k 421 us.)
// What bounds it: the LDS reads of operands and the vector unit that cuts fp32 into parts, a chunk's barriers
// between them.  A call with p = 64, r = 128, 160 heads of 4096 tokens: bf16 398-414 us, with the decay's gradient
// 732; fp32 732-756 and 1432.
#include "linear_scan.hpp"

namespace ssd {

// Kinds of work of a head's segment: the derivative along the decay (where `dots` are wanted), d_q, d_k, d_v,
// each in as many workgroups as its columns take.
template <class IO, int R, int P, bool WIDE, bool DECAY>
__global__ __launch_bounds__(256, 2) void k_linear_grad(LinearShape d, LinearGrads g) {
    using Keys = LinearScan<IO, P, kLinearTiles<IO, R, P>, 4, WIDE ? kWide : kOutputs>;  // d_q, d_k
    using Values = LinearScan<IO, R, kLinearTiles<IO, P, R>, 4, kOutputs>;
    using Tangent = LinearScan<IO, R, 1, 4, kTangent>;
    constexpr int KB = R <= Keys::PC ? 1 : R / Keys::PC, VB = P <= Values::PC ? 1 : P / Values::PC,
                  TB = !DECAY ? 0 : P <= Tangent::PC ? 1 : P / Tangent::PC, PER = TB + 2 * KB + VB;
    constexpr int L0 = Keys::LDS > Values::LDS ? Keys::LDS : Values::LDS;
    __shared__ __align__(16) char sm[DECAY && Tangent::LDS > L0 ? Tangent::LDS : L0];
    const int64_t blk = linear_order(blockIdx.x, gridDim.x), bh = blk / PER / d.segs;
    const int seg = static_cast<int>(blk / PER % d.segs);
    int at = static_cast<int>(blk % PER);
    if constexpr (DECAY) {
        if (at < TB) return Tangent(sm, d, g.decay, bh, seg, at * Tangent::PC).run();
        at -= TB;
    }
    if (at < 2 * KB) {
        LinearShape t = d;
        t.P = d.R;
        t.R = d.P;
        return Keys(sm, t, at < KB ? g.q : g.k, bh, seg, at % KB * Keys::PC).run();
    }
    Values(sm, d, g.v, bh, seg, (at - 2 * KB) * Values::PC).run();
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

// Workgroups that `width` columns take.
int blocks(int width, int tiles) { return width <= 64 * tiles ? 1 : width / (64 * tiles); }

template <class IO, int R, int P, bool WIDE, bool DECAY>
hipError_t grad(const LinearShape& d, const LinearGrads& g, hipStream_t st) {
    const int per = (DECAY ? blocks(P, 1) : 0) + 2 * blocks(R, kLinearTiles<IO, R, P>) + blocks(P, kLinearTiles<IO, P, R>);
    k_linear_grad<IO, R, P, WIDE, DECAY>
        <<<dim3(static_cast<unsigned>(static_cast<int64_t>(d.B) * d.H * d.segs * per)), 256, 0, st>>>(d, g);
    return hipGetLastError();
}

}  // namespace

int linear_grad_blocks(const LinearShape& d, bool decay) {
    auto of = [&](int columns, int rows) { return blocks(columns, linear_tiles(d.io == 1, columns, rows)); };
    return 2 * of(d.R, d.P) + of(d.P, d.R) + (decay ? blocks(d.P, 1) : 0);
}

hipError_t launch_linear_grad(const LinearShape& d, const LinearGrads& g, bool decay, hipStream_t st) {
    return by_widths(d.P, d.R, [&](auto p, auto r) {
        constexpr int P = decltype(p)::value, R = decltype(r)::value;
        auto go = [&](auto wide, auto dec) {
            constexpr bool W = decltype(wide)::value, D = decltype(dec)::value;
            if constexpr (!W)
                if (d.io == 0) return grad<F32, R, P, false, D>(d, g, st);
            return grad<BF16, R, P, W, D>(d, g, st);
        };
        const std::true_type yes;
        const std::false_type no;
        if (g.q.wide && d.io == 1) return decay ? go(yes, yes) : go(yes, no);  // (fp32 outputs are wide already)
        return decay ? go(no, yes) : go(no, no);
    });
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
