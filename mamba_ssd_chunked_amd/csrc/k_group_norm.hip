// Group norm over channels-last data with an activation or a gate.
//
// x [n, s, c], groups of c / groups neighbouring channels; mean and variance over the s positions and the
// channels of a group, of each sample:
//   m = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  u = m w + b,
//   y = u, silu(u), or u silu(gate).
// Gradient, with du the gradient of u and N the values of a group:
//   d_b = sum du,  d_w = sum du m  (over samples and positions, per channel),
//   d_x = rstd (w du - mean_N(w du) - m mean_N(w du m)),  d_gate = dy u silu'(gate).
//
// Where every position is a sample of its own (s = 1: tokens), a group's values lie side by side: a team
// of 1 to 64 lanes holds one in registers, and x is read once.  Otherwise a thread has one vector of EV
// channels for its whole life and walks down positions: one kernel leaves sums per block of positions,
// the next joins them, and a third writes the outputs, reading x again.  Variances are summed
// over runs of positions, about the thread's first value and then about its mean so far, and joined with the
// differences of the means: no square of a mean is subtracted, and of an outlier's distance from the run's mean
// only over the run.  No atomics: sums are joined in a fixed order.
// EV is the widest vector of 16 bytes or less that a group's channels divide into, or with positions a slab's of
// whole groups.
// Measured: 8192 tokens x 80 groups of 64 under a gate bf16 48 us (5.3 TB/s); 4 x 16384 positions x 512 channels with
// SiLU bf16 16 us for the statistics (4.2 TB/s), 3 to join them, 25 for the outputs (5.5 TB/s); 8192 tokens x 24
// groups of 64 fp32 under a gate 24 us (6.3 TB/s), their gradient 52-54 (5.0 TB/s) and 4.
#include <algorithm>
#include <type_traits>

#include "ssd_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {

namespace {

template <class IO, int EV>
__device__ __forceinline__ void ldv(const typename IO::T* p, float (&x)[EV]) {
    typedef typename IO::T vec __attribute__((ext_vector_type(EV)));
    if constexpr (sizeof(typename IO::T) == 4) {
        const vec w = *reinterpret_cast<const vec*>(p);
#pragma unroll
        for (int e = 0; e < EV; ++e) x[e] = w[e];
    } else if constexpr (EV == 1) {
        x[0] = bf16_to_f32(p[0]);
    } else {
        typedef uint32_t words __attribute__((ext_vector_type(EV / 2)));
        const words w = *reinterpret_cast<const words*>(p);
#pragma unroll
        for (int e = 0; e < EV / 2; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
}
template <class IO, int EV>
__device__ __forceinline__ void stv(typename IO::T* p, const float (&x)[EV]) {
    if constexpr (sizeof(typename IO::T) == 4) {
        typedef float vec __attribute__((ext_vector_type(EV)));
        vec w;
#pragma unroll
        for (int e = 0; e < EV; ++e) w[e] = x[e];
        *reinterpret_cast<vec*>(p) = w;
    } else if constexpr (EV == 1) {
        p[0] = f32_to_bf16(x[0]);
    } else {
        typedef uint32_t words __attribute__((ext_vector_type(EV / 2)));
        words w;
#pragma unroll
        for (int e = 0; e < EV / 2; ++e) w[e] = f32x2_to_bf16x2(x[2 * e], x[2 * e + 1]);
        *reinterpret_cast<words*>(p) = w;
    }
}
// weight or bias of EV channels, or `none` without one
template <int EV>
__device__ __forceinline__ void ld_chan(const float* p, int64_t at, float none, float (&x)[EV]) {
#pragma unroll
    for (int e = 0; e < EV; ++e) x[e] = none;
    if (p) {
        typedef float vec __attribute__((ext_vector_type(EV < 4 ? EV : 4)));
        constexpr int W = EV < 4 ? EV : 4;
#pragma unroll
        for (int m = 0; m < EV; m += W) {
            const vec w = *reinterpret_cast<const vec*>(p + at + m);
#pragma unroll
            for (int e = 0; e < W; ++e) x[m + e] = w[e];
        }
    }
}

// 1 / (1 + e^-x) from the hardware's base-2 exponential and reciprocal, about 1 ulp each.  The product
// with log2 e is carried to twice 24 bits: rounded once, it would cost |x| half steps of e^-x.  (With expf
// and a full division the outputs, not their bytes, bounded the kernels: 4 x 16384 positions x 512
// channels bf16 53 us.)
__device__ __forceinline__ float sigmoid(float x) {
    constexpr float kHi = -1.44269502162933349609375f, kLo = -1.92596303e-8f;  // -log2 e
    x = __builtin_amdgcn_fmed3f(x, -1.0e4f, 1.0e4f);  // 0 and 1 long before; beyond 2^127 / log2 e t would overflow
    const float t = x * kHi, lo = fmaf(x, kHi, -t) + x * kLo;
    // 2^lo = 1 + lo ln 2 to 24 bits: |lo| < 2^-16 where the power is neither 0 nor infinite, and those stay so
    return __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(t), fmaf(lo, 0.693147182f, 1.0f), 1.0f));
}

// The output for the normalised value m, and what its gradient needs.
struct Act {
    int act;
    bool gated;
    __device__ __forceinline__ float out(float u, float gate) const {
        return gated ? u * (gate * sigmoid(gate)) : act ? u * sigmoid(u) : u;
    }
    // the gradient of u for the gradient dy of the output; dg: that of the gate
    __device__ __forceinline__ float back(float dy, float u, float gate, float& dg) const {
        if (!gated && !act) return dy;
        const float z = gated ? gate : u, sg = sigmoid(z), rise = sg * (1.0f + z * (1.0f - sg));
        dg = dy * u * rise;
        return gated ? dy * (z * sg) : dy * rise;
    }
};

template <int TS>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
    for (int o = 1; o < TS; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

constexpr int MAXREC = 128;  // records of a group at most (cuts alone reach it)

}  // namespace

// ------------------------------------------------------------------ tokens: s = 1
// Teams of TS lanes with NV vectors each, a group a team.
template <class IO, int EV, int NV, int TS>
__global__ __launch_bounds__(256) void k_group_norm_rows(GroupShape d, const typename IO::T* __restrict__ x,
                                                         const float* __restrict__ weight,
                                                         const float* __restrict__ bias,
                                                         const typename IO::T* __restrict__ gate,
                                                         typename IO::T* __restrict__ y, float* __restrict__ stats) {
    constexpr int TEAMS = 256 / TS;
    const Act act{d.act, gate != nullptr};
    const int lane = threadIdx.x % TS;
    const int64_t teams = d.n * d.groups;
    for (int64_t team = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TS; team < teams;
         team += static_cast<int64_t>(gridDim.x) * TEAMS) {
        const int64_t row = team / d.groups;
        const int ch = static_cast<int>(team % d.groups) * d.cg;
        float v[NV][EV], w[NV][EV], b[NV][EV], z[NV][EV];
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int col = (lane + m * TS) * EV;
            if (col < d.cg) {
                ldv<IO, EV>(x + row * d.x_stride + ch + col, v[m]);
                if (gate) ldv<IO, EV>(gate + row * d.gate_stride + ch + col, z[m]);
                ld_chan<EV>(weight, ch + col, 1.0f, w[m]);
                ld_chan<EV>(bias, ch + col, 0.0f, b[m]);
            }
        }
        // about the group's first value: exact for a constant group, and no sum of large means is rounded
        const float first = __shfl(v[0][0], 0, TS);
        float sum = 0.0f;
#pragma unroll
        for (int m = 0; m < NV; ++m)
            if ((lane + m * TS) * EV < d.cg) {
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    v[m][e] -= first;
                    sum += v[m][e];
                }
            }
        const float mean = team_sum<TS>(sum) * d.inv_count;
        float sq = 0.0f;
#pragma unroll
        for (int m = 0; m < NV; ++m)
            if ((lane + m * TS) * EV < d.cg) {
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    v[m][e] -= mean;
                    sq += v[m][e] * v[m][e];
                }
            }
        const float rstd = 1.0f / sqrtf(team_sum<TS>(sq) * d.inv_count + d.eps);
        if (stats && lane == 0) {
            stats[2 * team] = first + mean;
            stats[2 * team + 1] = rstd;
        }
        if (y) {
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const int col = (lane + m * TS) * EV;
                if (col < d.cg) {
#pragma unroll
                    for (int e = 0; e < EV; ++e)
                        v[m][e] = act.out(v[m][e] * rstd * w[m][e] + b[m][e], gate ? z[m][e] : 0.0f);
                    stv<IO, EV>(y + row * d.c + ch + col, v[m]);
                }
            }
        }
    }
}

// Team slot t of a workgroup keeps its group and walks down the rows; part [rows' parts, 2, c] holds what
// each leaves of d_weight and d_bias.
template <class IO, int EV, int NV, int TS>
__global__ __launch_bounds__(256) void k_group_norm_rows_bwd(
    GroupShape d, const typename IO::T* __restrict__ dy, const typename IO::T* __restrict__ x,
    const float* __restrict__ weight, const float* __restrict__ bias, const typename IO::T* __restrict__ gate,
    const float* __restrict__ stats, typename IO::T* __restrict__ d_x, typename IO::T* __restrict__ d_gate,
    float* __restrict__ part) {
    const Act act{d.act, gate != nullptr};
    const int lane = threadIdx.x % TS, slot = threadIdx.x / TS;
    const int slab = static_cast<int>(blockIdx.x % d.sums.slabs), block = static_cast<int>(blockIdx.x / d.sums.slabs);
    const int g = slab * d.sums.slab_groups + slot % d.sums.slab_groups, rl = slot / d.sums.slab_groups;
    if (rl >= d.sums.lanes || g >= d.groups) return;  // a whole team
    const int64_t p = static_cast<int64_t>(block) * d.sums.lanes + rl, parts = static_cast<int64_t>(d.sums.blocks) * d.sums.lanes;
    const int ch = g * d.cg;
    float w[NV][EV], b[NV][EV], dw[NV][EV], db[NV][EV];
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int col = (lane + m * TS) * EV;
        if (col < d.cg) {
            ld_chan<EV>(weight, ch + col, 1.0f, w[m]);
            ld_chan<EV>(bias, ch + col, 0.0f, b[m]);
        }
#pragma unroll
        for (int e = 0; e < EV; ++e) dw[m][e] = db[m][e] = 0.0f;
    }
    for (int64_t row = p; row < d.n; row += parts) {
        const float mean = stats[2 * (row * d.groups + g)], rstd = stats[2 * (row * d.groups + g) + 1];
        float v[NV][EV], du[NV][EV];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int col = (lane + m * TS) * EV;
            if (col < d.cg) {
                float z[EV], dg[EV];
                ldv<IO, EV>(x + row * d.x_stride + ch + col, v[m]);
                ldv<IO, EV>(dy + row * d.c + ch + col, du[m]);
                if (gate) ldv<IO, EV>(gate + row * d.gate_stride + ch + col, z);
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    v[m][e] = (v[m][e] - mean) * rstd;
                    du[m][e] = act.back(du[m][e], v[m][e] * w[m][e] + b[m][e], gate ? z[e] : 0.0f, dg[e]);
                    dw[m][e] += du[m][e] * v[m][e];
                    db[m][e] += du[m][e];
                    du[m][e] *= w[m][e];
                    s1 += du[m][e];
                    s2 += du[m][e] * v[m][e];
                }
                if (gate) stv<IO, EV>(d_gate + row * d.c + ch + col, dg);
            }
        }
        s1 = team_sum<TS>(s1) * d.inv_count;
        s2 = team_sum<TS>(s2) * d.inv_count;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int col = (lane + m * TS) * EV;
            if (col < d.cg) {
#pragma unroll
                for (int e = 0; e < EV; ++e) v[m][e] = rstd * (du[m][e] - s1 - v[m][e] * s2);
                stv<IO, EV>(d_x + row * d.c + ch + col, v[m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int col = (lane + m * TS) * EV;
        if (col < d.cg) {
            stv<F32, EV < 4 ? EV : 4>(part + (2 * p) * d.c + ch + col, *reinterpret_cast<float(*)[EV < 4 ? EV : 4]>(dw[m]));
            stv<F32, EV < 4 ? EV : 4>(part + (2 * p + 1) * d.c + ch + col,
                                      *reinterpret_cast<float(*)[EV < 4 ? EV : 4]>(db[m]));
            if constexpr (EV == 8) {
                stv<F32, 4>(part + (2 * p) * d.c + ch + col + 4, *reinterpret_cast<float(*)[4]>(dw[m] + 4));
                stv<F32, 4>(part + (2 * p + 1) * d.c + ch + col + 4, *reinterpret_cast<float(*)[4]>(db[m] + 4));
            }
        }
    }
}

// ------------------------------------------------------------------ positions: s > 1, or wide groups
namespace {

// A workgroup's piece: a block of the positions of one sample, and a slab of channels: whole groups, or
// one of the `cuts` parts of a group wider than 256 vectors.  Thread t has the vector t % cv of the
// slab's, and every lanes-th position from t / cv on.  A vector may reach over groups.
template <int EV>
struct Piece {
    int64_t n, r0, r1;
    int block, g0, ng, cut, ch0, nch, cv, col, rl, lanes;
    bool on;
    __device__ Piece(const GroupShape& d, const GroupCut& c, int64_t item) {
        const int slab = static_cast<int>(item % c.slabs);
        block = static_cast<int>(item / c.slabs % c.blocks);
        n = item / c.slabs / c.blocks;
        lanes = c.lanes;
        if (c.cuts == 1) {
            cut = 0;
            g0 = slab * c.slab_groups;
            ng = d.groups - g0 < c.slab_groups ? d.groups - g0 : c.slab_groups;
            ch0 = g0 * d.cg;
            nch = ng * d.cg;
            cv = c.slab_groups * d.cg / EV;
        } else {
            cut = slab % c.cuts;
            g0 = slab / c.cuts;
            ng = 1;
            ch0 = g0 * d.cg + cut * 256 * EV;
            nch = d.cg - cut * 256 * EV < 256 * EV ? d.cg - cut * 256 * EV : 256 * EV;
            cv = 256;
        }
        col = threadIdx.x % cv;
        rl = threadIdx.x / cv;
        on = rl < lanes && col * EV < nch;
        r0 = static_cast<int64_t>(block) * c.rows;
        r1 = r0 + c.rows < d.s ? r0 + c.rows : d.s;
    }
    __device__ int channel() const { return ch0 + col * EV; }
};

// Positions that row lane rl of `lanes` has of those in [r0, r1).
__device__ __forceinline__ int64_t lane_rows(int64_t r0, int64_t r1, int rl, int lanes) {
    return r0 + rl < r1 ? (r1 - r0 - rl + lanes - 1) / lanes : 0;
}

}  // namespace

namespace {

// Positions of a run whose sums are taken about one value.  Where that is an outlier, D from the rest, the two
// sums of a run of N are N D^2 and leave D^2: an error that grows with N and, over a thousand positions, reached
// 7e-4 of the variance.
constexpr int RUN = 32;

// Mean and sum of squared differences of a piece's groups over its positions: f(group of the slab, mean,
// squares) in one lane.  sh: free again after the next barrier.
template <class IO, int EV, class F>
__device__ __forceinline__ void piece_moments(const GroupShape& d, const Piece<EV>& p, const typename IO::T* x,
                                              float2 (&sh)[EV][256], F&& f) {
    float mean[EV], m2[EV];
#pragma unroll
    for (int e = 0; e < EV; ++e) mean[e] = m2[e] = 0.0f;
    if (p.on && p.r0 + p.rl < p.r1) {
        const typename IO::T* at = x + (p.n * d.s + p.r0 + p.rl) * d.x_stride + p.channel();
        float about[EV];
        ldv<IO, EV>(at, about);
        const int64_t rows = lane_rows(p.r0, p.r1, p.rl, p.lanes), step = p.lanes * d.x_stride;
        constexpr int WAY = EV > 2 ? 8 : 16;  // loads under way (7000 positions x 4099 fp32 channels: 8 127 us, 16 110)
        // of the runs so far: the mean is about + low
        float low[EV], sq[EV];
#pragma unroll
        for (int e = 0; e < EV; ++e) low[e] = sq[e] = 0.0f;
        for (int64_t done = 0; done < rows; done += RUN) {
            const int n = static_cast<int>(rows - done < RUN ? rows - done : RUN);
            float s1[EV], s2[EV];
#pragma unroll
            for (int e = 0; e < EV; ++e) s1[e] = s2[e] = 0.0f;
            for (int r = 0; r < n; r += WAY) {  // past the last position that one again
                float v[WAY][EV];
#pragma unroll
                for (int m = 0; m < WAY; ++m) ldv<IO, EV>(at + (done + (r + m < n ? r + m : n - 1)) * step, v[m]);
#pragma unroll
                for (int m = 0; m < WAY; ++m)
#pragma unroll
                    for (int e = 0; e < EV; ++e) {
                        const float o = r + m < n ? v[m][e] - about[e] : 0.0f;
                        s1[e] += o;
                        s2[e] += o * o;
                    }
            }
            const float inv = 1.0f / static_cast<float>(n), all = static_cast<float>(done + n),
                        share = done ? static_cast<float>(n) / all : 1.0f;
#pragma unroll
            for (int e = 0; e < EV; ++e) {
                const float off = s1[e] * inv, gap = off - low[e], on = low[e] + gap * share, was = about[e];
                sq[e] += fmaxf(s2[e] - s1[e] * off, 0.0f);
                if (done) sq[e] += gap * gap * (share * static_cast<float>(done));
                about[e] += on;
                low[e] = on - (about[e] - was);  // (what the sum rounds off, however many runs)
            }
        }
        const float cnt = static_cast<float>(rows);
#pragma unroll
        for (int e = 0; e < EV; ++e) {
            mean[e] = about[e];
            m2[e] = sq[e];
        }
        // channels of one group, `sub` at a time, by halves of equal counts
#pragma unroll
        for (int wide = 1; wide < EV; wide *= 2)
            if (wide < d.sub) {
#pragma unroll
                for (int e = 0; e < EV; e += 2 * wide) {
                    const float off = mean[e + wide] - mean[e];
                    m2[e] += m2[e + wide] + off * off * (0.5f * cnt * static_cast<float>(wide));
                    mean[e] += 0.5f * off;
                }
            }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EV; ++e) sh[e][threadIdx.x] = make_float2(mean[e], m2[e]);
    __syncthreads();
    // per group: its records of every row lane, joined by a power of two of lanes.  Means are averaged as
    // differences from one of them: exactly for a constant group, and else without roundings of the mean's size.
    const int per = p.nch / (p.ng * d.sub), R = static_cast<int>(p.r1 - p.r0), base = R / p.lanes, more = R % p.lanes;
    const float total = static_cast<float>(R) * static_cast<float>(per * d.sub);
    int lanes = 64;
    while (lanes > 8 && lanes * p.ng > 256) lanes /= 2;
    auto team = [&](float v) {
        for (int o = 1; o < lanes; o <<= 1) v += __shfl_xor(v, o);
        return v;
    };
    const int l = threadIdx.x % lanes;
    for (int g = threadIdx.x / lanes; g < p.ng; g += 256 / lanes) {
        auto each = [&](auto&& f) {
            float sum = 0.0f;
            for (int k = l; k < p.lanes * per; k += lanes) {
                const int rl = k / per, c = (g * per + k - rl * per) * d.sub;
                sum += f(sh[c % EV][rl * p.cv + c / EV], static_cast<float>((base + (rl < more)) * d.sub));
            }
            return team(sum);
        };
        const float one = sh[g * per * d.sub % EV][g * per * d.sub / EV].x;  // the group's first record's
        const float mu = one + each([&](float2 r, float cnt) { return cnt * (r.x - one); }) / total;
        const float sum = each([&](float2 r, float cnt) { return r.y + cnt * (r.x - mu) * (r.x - mu); });
        if (l == 0) f(g, mu, sum);
    }
}

// y of a piece; stat(group): its mean and 1 / sqrt(var + eps).
template <class IO, int EV, class F>
__device__ __forceinline__ void piece_outputs(const GroupShape& d, const Piece<EV>& p, const typename IO::T* x,
                                              const float* weight, const float* bias, const typename IO::T* gate,
                                              F&& stat, typename IO::T* y) {
    if (!p.on) return;
    const Act act{d.act, gate != nullptr};
    const int ch = p.channel();
    float mean[EV], w[EV], b[EV];
    ld_chan<EV>(weight, ch, 1.0f, w);
    ld_chan<EV>(bias, ch, 0.0f, b);
#pragma unroll
    for (int e = 0; e < EV; ++e) {
        const float2 t = stat((ch + e) / d.cg);
        mean[e] = t.x;
        w[e] *= t.y;
    }
#pragma unroll 4
    for (int64_t r = p.r0 + p.rl; r < p.r1; r += p.lanes) {
        const int64_t row = p.n * d.s + r;
        float v[EV], z[EV];
        ldv<IO, EV>(x + row * d.x_stride + ch, v);
        if (gate) ldv<IO, EV>(gate + row * d.gate_stride + ch, z);
#pragma unroll
        for (int e = 0; e < EV; ++e) v[e] = act.out((v[e] - mean[e]) * w[e] + b[e], gate ? z[e] : 0.0f);
        stv<IO, EV>(y + row * d.c + ch, v);
    }
}

}  // namespace

// Everything of a slab's groups of one sample.
template <class IO, int EV>
__global__ __launch_bounds__(256) void k_group_norm_whole(GroupShape d, const typename IO::T* __restrict__ x,
                                                          const float* __restrict__ weight,
                                                          const float* __restrict__ bias,
                                                          const typename IO::T* __restrict__ gate,
                                                          typename IO::T* __restrict__ y, float* __restrict__ stats) {
    __shared__ float2 sh[EV][256], st[256];
    const int64_t items = d.n * d.sums.slabs;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const Piece<EV> p(d, d.sums, item);
        piece_moments<IO, EV>(d, p, x, sh, [&](int g, float mu, float sum) {
            st[g] = make_float2(mu, 1.0f / sqrtf(sum * d.inv_count + d.eps));
            if (stats) reinterpret_cast<float2*>(stats)[p.n * d.groups + p.g0 + g] = st[g];
        });
        __syncthreads();
        if (y) piece_outputs<IO, EV>(d, p, x, weight, bias, gate, [&](int g) { return st[g - p.g0]; }, y);
    }
}

// Mean and sum of squared differences of every (sample, group, block of positions, cut):
// rec [n, groups, blocks, cuts].
template <class IO, int EV>
__global__ __launch_bounds__(256) void k_group_norm_stats(GroupShape d, const typename IO::T* __restrict__ x,
                                                          float2* __restrict__ rec) {
    __shared__ float2 sh[EV][256];
    const int64_t items = d.n * d.sums.blocks * d.sums.slabs;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const Piece<EV> p(d, d.sums, item);
        piece_moments<IO, EV>(d, p, x, sh, [&](int g, float mu, float sum) {
            rec[((p.n * d.groups + p.g0 + g) * d.sums.blocks + p.block) * d.sums.cuts + p.cut] = make_float2(mu, sum);
        });
    }
}

// The statistics of a (sample, group) from its records, a wave each.
__global__ __launch_bounds__(256) void k_group_norm_join(GroupShape d, const float2* __restrict__ rec,
                                                         float2* __restrict__ stats) {
    const int K = d.sums.blocks * d.sums.cuts, l = threadIdx.x & 63;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); at < d.n * d.groups;
         at += static_cast<int64_t>(gridDim.x) * 4) {
        const float one = rec[at * K].x;
        float2 r[MAXREC / 64];
        float cnt[MAXREC / 64], sum = 0.0f;
#pragma unroll
        for (int m = 0; m < MAXREC / 64; ++m) {
            const int k = l + m * 64;
            r[m] = make_float2(0.0f, 0.0f);
            cnt[m] = 0.0f;
            if (k < K) {
                r[m] = rec[at * K + k];
                const int64_t r0 = static_cast<int64_t>(k / d.sums.cuts) * d.sums.rows;
                const int wide = d.cg - k % d.sums.cuts * 256 * d.ev;
                cnt[m] = static_cast<float>((r0 + d.sums.rows < d.s ? d.sums.rows : d.s - r0) *
                                            (d.sums.cuts > 1 && wide > 256 * d.ev ? 256 * d.ev : wide));
            }
            sum += cnt[m] * (r[m].x - one);
        }
        const float mu = one + team_sum<64>(sum) * d.inv_count;
        sum = 0.0f;
#pragma unroll
        for (int m = 0; m < MAXREC / 64; ++m) sum += r[m].y + cnt[m] * (r[m].x - mu) * (r[m].x - mu);
        sum = team_sum<64>(sum);
        if (l == 0) stats[at] = make_float2(mu, 1.0f / sqrtf(sum * d.inv_count + d.eps));
    }
}

template <class IO, int EV>
__global__ __launch_bounds__(256) void k_group_norm_apply(GroupShape d, const typename IO::T* __restrict__ x,
                                                          const float* __restrict__ weight,
                                                          const float* __restrict__ bias,
                                                          const typename IO::T* __restrict__ gate,
                                                          const float2* __restrict__ stats,
                                                          typename IO::T* __restrict__ y) {
    const int64_t items = d.n * d.outs.blocks * d.outs.slabs;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const Piece<EV> p(d, d.outs, item);
        piece_outputs<IO, EV>(d, p, x, weight, bias, gate, [&](int g) { return stats[p.n * d.groups + g]; }, y);
    }
}

// Per channel, the sums of du and du m over a block of positions: part [n, blocks, 2, c].
template <class IO, int EV>
__global__ __launch_bounds__(256) void k_group_norm_sums(GroupShape d, const typename IO::T* __restrict__ dy,
                                                         const typename IO::T* __restrict__ x,
                                                         const float* __restrict__ weight,
                                                         const float* __restrict__ bias,
                                                         const typename IO::T* __restrict__ gate,
                                                         const float* __restrict__ stats, float* __restrict__ part) {
    __shared__ float sh[2 * EV][256];
    const Act act{d.act, gate != nullptr};
    const int64_t items = d.n * d.sums.blocks * d.sums.slabs;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const Piece<EV> p(d, d.sums, item);
        float s1[EV], s2[EV];
#pragma unroll
        for (int e = 0; e < EV; ++e) s1[e] = s2[e] = 0.0f;
        if (p.on) {
            const int ch = p.channel();
            float w[EV], b[EV], mean[EV], rstd[EV];
            ld_chan<EV>(weight, ch, 1.0f, w);
            ld_chan<EV>(bias, ch, 0.0f, b);
#pragma unroll
            for (int e = 0; e < EV; ++e) {
                const float2 st = reinterpret_cast<const float2*>(stats)[p.n * d.groups + (ch + e) / d.cg];
                mean[e] = st.x;
                rstd[e] = st.y;
            }
#pragma unroll 4
            for (int64_t r = p.r0 + p.rl; r < p.r1; r += p.lanes) {
                const int64_t row = p.n * d.s + r;
                float v[EV], g[EV], z[EV], dg;
                ldv<IO, EV>(x + row * d.x_stride + ch, v);
                ldv<IO, EV>(dy + row * d.c + ch, g);
                if (gate) ldv<IO, EV>(gate + row * d.gate_stride + ch, z);
#pragma unroll
                for (int e = 0; e < EV; ++e) {
                    const float m = (v[e] - mean[e]) * rstd[e];
                    const float du = act.back(g[e], m * w[e] + b[e], gate ? z[e] : 0.0f, dg);
                    s1[e] += du;
                    s2[e] += du * m;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < EV; ++e) {
            sh[e][threadIdx.x] = s1[e];
            sh[EV + e][threadIdx.x] = s2[e];
        }
        __syncthreads();
        for (int k = threadIdx.x; k < 2 * p.nch; k += 256) {
            const int which = k >= p.nch, c = k - which * p.nch;
            double sum = 0.0;
            for (int l = 0; l < p.lanes; ++l) sum += sh[which * EV + c % EV][l * p.cv + c / EV];
            part[((p.n * d.sums.blocks + p.block) * 2 + which) * d.c + p.ch0 + c] = static_cast<float>(sum);
        }
    }
}

// Joins the blocks of a (sample, group): chan [n, 2, c] = sums per channel, mean [n, groups] the means of
// w du and w du m over the group.
__global__ __launch_bounds__(256) void k_group_norm_means(GroupShape d, const float* __restrict__ part,
                                                          const float* __restrict__ weight, float* __restrict__ chan,
                                                          float2* __restrict__ mean) {
    __shared__ double sh[2][256];
    int cw = 1;  // channels at a time, as many lanes as are left for each
    while (cw < d.cg && cw < 256) cw *= 2;
    const int lanes = 256 / cw, lc = threadIdx.x % cw, bl = threadIdx.x / cw;
    for (int64_t item = blockIdx.x; item < d.n * d.groups; item += gridDim.x) {
        const int64_t n = item / d.groups;
        const int g = static_cast<int>(item % d.groups);
        float s1 = 0.0f, s2 = 0.0f;
        for (int c0 = 0; c0 < d.cg; c0 += cw) {
            const int c = c0 + lc, ch = g * d.cg + c;
            double a = 0.0, b = 0.0;
            if (c < d.cg) {
#pragma unroll 4
                for (int k = bl; k < d.sums.blocks; k += lanes) {
                    a += part[((n * d.sums.blocks + k) * 2) * d.c + ch];
                    b += part[((n * d.sums.blocks + k) * 2 + 1) * d.c + ch];
                }
            }
            __syncthreads();
            sh[0][threadIdx.x] = a;
            sh[1][threadIdx.x] = b;
            __syncthreads();
            if (bl == 0 && c < d.cg) {
                for (int l = 1; l < lanes; ++l) {
                    a += sh[0][l * cw + lc];
                    b += sh[1][l * cw + lc];
                }
                const float w = weight ? weight[ch] : 1.0f, du = static_cast<float>(a), dum = static_cast<float>(b);
                chan[(2 * n) * d.c + ch] = dum;
                chan[(2 * n + 1) * d.c + ch] = du;
                s1 += w * du;
                s2 += w * dum;
            }
        }
        s1 = team_sum<64>(s1);
        s2 = team_sum<64>(s2);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
            sh[0][threadIdx.x >> 6] = s1;
            sh[1][threadIdx.x >> 6] = s2;
        }
        __syncthreads();
        if (threadIdx.x == 0)
            mean[item] = make_float2(static_cast<float>(sh[0][0] + sh[0][1] + sh[0][2] + sh[0][3]) * d.inv_count,
                                     static_cast<float>(sh[1][0] + sh[1][1] + sh[1][2] + sh[1][3]) * d.inv_count);
    }
}

// d_x and d_gate of the pieces; the first workgroups have d_weight and d_bias [c], 32 channels each, the sums
// over samples of chan.
template <class IO, int EV>
__global__ __launch_bounds__(256) void k_group_norm_grad(GroupShape d, const typename IO::T* __restrict__ dy,
                                                         const typename IO::T* __restrict__ x,
                                                         const float* __restrict__ weight,
                                                         const float* __restrict__ bias,
                                                         const typename IO::T* __restrict__ gate,
                                                         const float* __restrict__ stats,
                                                         const float2* __restrict__ mean,
                                                         typename IO::T* __restrict__ d_x,
                                                         typename IO::T* __restrict__ d_gate,
                                                         const float* __restrict__ chan, int sums,
                                                         float* __restrict__ d_weight, float* __restrict__ d_bias) {
    __shared__ double sh[8][33];
    const Act act{d.act, gate != nullptr};
    if (static_cast<int>(blockIdx.x) < sums) {
        const int l = threadIdx.x & 31, run = threadIdx.x >> 5, which = blockIdx.x & 1, col = (blockIdx.x >> 1) * 32 + l;
        float* to = which ? d_bias : d_weight;
        double acc = 0.0;
        if (col < d.c) {
#pragma unroll 8  // as many loads under way
            for (int64_t n = run; n < d.n; n += 8) acc += chan[(2 * n + which) * d.c + col];
        }
        sh[run][l] = acc;
        __syncthreads();
        if (run == 0 && col < d.c && to) {
            for (int m = 1; m < 8; ++m) acc += sh[m][l];
            to[col] = static_cast<float>(acc);
        }
        return;
    }
    const int64_t items = d.n * d.outs.blocks * d.outs.slabs;
    for (int64_t item = blockIdx.x - sums; item < items; item += gridDim.x - sums) {
        const Piece<EV> p(d, d.outs, item);
        if (!p.on) continue;
        const int ch = p.channel();
        float w[EV], b[EV], mu[EV], rstd[EV], m1[EV], m2[EV];
        ld_chan<EV>(weight, ch, 1.0f, w);
        ld_chan<EV>(bias, ch, 0.0f, b);
#pragma unroll
        for (int e = 0; e < EV; ++e) {
            const int64_t at = p.n * d.groups + (ch + e) / d.cg;
            const float2 st = reinterpret_cast<const float2*>(stats)[at], mn = mean[at];
            mu[e] = st.x;
            rstd[e] = st.y;
            m1[e] = mn.x;
            m2[e] = mn.y;
        }
#pragma unroll 4
        for (int64_t r = p.r0 + p.rl; r < p.r1; r += p.lanes) {
            const int64_t row = p.n * d.s + r;
            float v[EV], g[EV], z[EV], dg[EV];
            ldv<IO, EV>(x + row * d.x_stride + ch, v);
            ldv<IO, EV>(dy + row * d.c + ch, g);
            if (gate) ldv<IO, EV>(gate + row * d.gate_stride + ch, z);
#pragma unroll
            for (int e = 0; e < EV; ++e) {
                const float m = (v[e] - mu[e]) * rstd[e];
                const float du = act.back(g[e], m * w[e] + b[e], gate ? z[e] : 0.0f, dg[e]);
                v[e] = rstd[e] * (w[e] * du - m1[e] - m * m2[e]);
            }
            stv<IO, EV>(d_x + row * d.c + ch, v);
            if (gate) stv<IO, EV>(d_gate + row * d.c + ch, dg);
        }
    }
}

// d_weight, d_bias [c] = sums over parts of part [parts, 2, c]: 32 columns x 32 interleaved runs of parts.
__global__ __launch_bounds__(1024) void k_group_norm_weight(const float* __restrict__ part, int64_t parts, int c,
                                                            float* __restrict__ d_weight, float* __restrict__ d_bias) {
    __shared__ double sh[32][33];
    const int l = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int col = static_cast<int>(blockIdx.x) * 32 + l;
    float* to = blockIdx.y ? d_bias : d_weight;
    if (!to) return;
    double acc = 0.0;
    if (col < c) {
#pragma unroll 8  // as many loads under way
        for (int64_t t = run; t < parts; t += 32) acc += part[(2 * t + blockIdx.y) * c + col];
    }
    sh[run][l] = acc;
    __syncthreads();
    if (run == 0 && col < c) {
        acc = 0.0;
#pragma unroll
        for (int m = 0; m < 32; ++m) acc += sh[m][l];
        to[col] = static_cast<float>(acc);
    }
}

namespace {

constexpr int64_t kMaxGroups = 1 << 20;  // workgroups of a launch; more work goes round in it
unsigned grid_of(int64_t items) { return static_cast<unsigned>(items < kMaxGroups ? items : kMaxGroups); }

template <class IO, class F>
hipError_t by_vector(const GroupShape& d, F&& f) {
    if constexpr (sizeof(typename IO::T) == 2)
        if (d.ev == 8) return f(std::integral_constant<int, 8>{});
    if (d.ev == 4) return f(std::integral_constant<int, 4>{});
    if (d.ev == 2) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
}
// The smallest team whose lanes hold a vector each; 64 lanes with up to eight for wider groups.
template <class F>
hipError_t by_team(int cgv, F&& f) {
    const std::integral_constant<int, 1> one;
    if (cgv <= 1) return f(one, std::integral_constant<int, 1>{});
    if (cgv <= 2) return f(one, std::integral_constant<int, 2>{});
    if (cgv <= 4) return f(one, std::integral_constant<int, 4>{});
    if (cgv <= 8) return f(one, std::integral_constant<int, 8>{});
    if (cgv <= 16) return f(one, std::integral_constant<int, 16>{});
    if (cgv <= 32) return f(one, std::integral_constant<int, 32>{});
    const std::integral_constant<int, 64> wave;
    if (cgv <= 64) return f(one, wave);
    if (cgv <= 128) return f(std::integral_constant<int, 2>{}, wave);
    if (cgv <= 256) return f(std::integral_constant<int, 4>{}, wave);
    return f(std::integral_constant<int, 8>{}, wave);
}
int team_of(int cgv) {
    int t = 1;
    while (t < cgv && t < 64) t *= 2;
    return t;
}

template <class F>
hipError_t by_io(const GroupShape& d, F&& f) {
    return d.io == 1 ? f(BF16{}) : f(F32{});
}

}  // namespace

// Positions or tokens whose terms a thread of the gradient adds up in fp32: of one sign and size their roundings go to
// one side, half of such a step for each in the end (1e-5 of the sum over 1000, 4e-5 over 4000).  The rest goes in fp64.
constexpr int64_t kMaxRun = 256;

// Which way, and how the work is cut up.
void group_norm_plan(GroupShape* d, bool bwd) {
    // blocks of `rows` over `lanes` by which a thread has no more than kMaxRun of them (as far as a launch goes)
    auto short_runs = [](int64_t rows, int64_t lanes, int64_t slabs) {
        return std::min((rows + kMaxRun * lanes - 1) / (kMaxRun * lanes), std::max<int64_t>(kMaxGroups / slabs, 1));
    };
    const int V = d->io == 1 ? 8 : 4;
    auto widest = [&](int of) {
        int ev = V;
        while (of % ev || d->x_stride % ev || d->gate_stride % ev) ev /= 2;
        return ev;
    };
    d->ev = widest(d->cg);
    const int cgv = d->cg / d->ev;
    d->tokens = d->s == 1 && cgv <= 512;
    if (d->tokens) {
        if (!bwd) return;
        GroupCut& c = d->sums;
        const int teams = 256 / team_of(cgv);
        c.slab_groups = d->groups < teams ? d->groups : teams;
        c.lanes = teams / c.slab_groups;
        c.slabs = (d->groups + c.slab_groups - 1) / c.slab_groups;
        int64_t b = 2048 / c.slabs;
        const int64_t most = (d->n + c.lanes - 1) / c.lanes;
        if (b > 1024 / c.lanes) b = 1024 / c.lanes;
        b = std::max(b, short_runs(d->n, c.lanes, c.slabs));
        if (b > most) b = most;
        c.blocks = static_cast<int>(b < 1 ? 1 : b);
        return;
    }
    // vectors that reach over groups, where a slab of whole groups is whole vectors (ten channels of
    // bf16: vectors of eight over slabs of a multiple of four groups)
    const int wide = widest(d->c);
    int unit = 1;  // groups of whole vectors
    while (unit * d->cg % wide) unit *= 2;
    if (wide > d->ev && unit * d->cg / wide <= 256)
        d->ev = wide;
    else
        unit = 1;
    d->sub = 1;
    while (2 * d->sub <= d->ev && d->cg % (2 * d->sub) == 0) d->sub *= 2;
    const int unit_vectors = unit * d->cg / d->ev;
    auto cut = [&](int units, int each, int most, bool runs) {
        GroupCut c{};
        c.cuts = unit_vectors > 256 ? (unit_vectors + 255) / 256 : 1;
        c.slab_groups = units < 2 ? unit : units * unit;
        if (c.slab_groups > 256) c.slab_groups = 256;  // (a whole number of units, at most eight groups)
        if (c.slab_groups > d->groups) c.slab_groups = d->groups;
        c.slabs = (d->groups + c.slab_groups - 1) / c.slab_groups * c.cuts;
        c.lanes = c.cuts > 1 ? 1 : 256 / (c.slab_groups * d->cg / d->ev);
        // blocks of positions: workgroups for the chip, at least `each` positions a thread
        int64_t b = 2048 / (d->n * c.slabs);
        const int64_t whole = (d->s + each * c.lanes - 1) / (each * c.lanes);
        if (b > most / c.cuts) b = most / c.cuts;
        if (b > whole) b = whole;
        if (b < 1) b = 1;
        if (runs) b = std::max(b, short_runs(d->s, c.lanes, c.slabs));
        c.rows = (d->s + b - 1) / b;
        c.blocks = static_cast<int>((d->s + c.rows - 1) / c.rows);
        return c;
    };
    // sums: about 256 bytes of neighbouring channels, which leave many positions to a workgroup and few
    // records to a group; outputs: whole rows
    d->sums = cut((15 + unit_vectors) / unit_vectors, 8, MAXREC, bwd);
    d->outs = cut(256 / unit_vectors, 4, 1 << 20, false);
    d->whole = d->sums.blocks == 1 && d->sums.cuts == 1;
}

hipError_t launch_group_norm(const GroupShape& d, const void* x, const float* weight, const float* bias,
                             const void* gate, void* y, float* stats, hipStream_t st) {
    return by_io(d, [&](auto io_) {
        using IO = decltype(io_);
        using T = typename IO::T;
        return by_vector<IO>(d, [&](auto ev) {
            constexpr int EV = decltype(ev)::value;
            return by_team(d.cg / EV, [&](auto nv, auto ts) {
                constexpr int NV = decltype(nv)::value, TS = decltype(ts)::value;
                const int64_t per = 256 / TS;
                k_group_norm_rows<IO, EV, NV, TS><<<grid_of((d.n * d.groups + per - 1) / per), 256, 0, st>>>(
                    d, static_cast<const T*>(x), weight, bias, static_cast<const T*>(gate), static_cast<T*>(y), stats);
                return hipGetLastError();
            });
        });
    });
}

hipError_t launch_group_norm_whole(const GroupShape& d, const void* x, const float* weight, const float* bias,
                                   const void* gate, void* y, float* stats, hipStream_t st) {
    return by_io(d, [&](auto io_) {
        using IO = decltype(io_);
        using T = typename IO::T;
        return by_vector<IO>(d, [&](auto ev) {
            k_group_norm_whole<IO, decltype(ev)::value><<<grid_of(d.n * d.sums.slabs), 256, 0, st>>>(
                d, static_cast<const T*>(x), weight, bias, static_cast<const T*>(gate), static_cast<T*>(y), stats);
            return hipGetLastError();
        });
    });
}

hipError_t launch_group_norm_stats(const GroupShape& d, const void* x, float* rec, hipStream_t st) {
    return by_io(d, [&](auto io_) {
        using IO = decltype(io_);
        return by_vector<IO>(d, [&](auto ev) {
            k_group_norm_stats<IO, decltype(ev)::value><<<grid_of(d.n * d.sums.blocks * d.sums.slabs), 256, 0, st>>>(
                d, static_cast<const typename IO::T*>(x), reinterpret_cast<float2*>(rec));
            return hipGetLastError();
        });
    });
}

hipError_t launch_group_norm_join(const GroupShape& d, const float* rec, float* stats, hipStream_t st) {
    k_group_norm_join<<<grid_of((d.n * d.groups + 3) / 4), 256, 0, st>>>(d, reinterpret_cast<const float2*>(rec),
                                                                         reinterpret_cast<float2*>(stats));
    return hipGetLastError();
}

hipError_t launch_group_norm_apply(const GroupShape& d, const void* x, const float* weight, const float* bias,
                                   const void* gate, const float* stats, void* y, hipStream_t st) {
    return by_io(d, [&](auto io_) {
        using IO = decltype(io_);
        using T = typename IO::T;
        return by_vector<IO>(d, [&](auto ev) {
            k_group_norm_apply<IO, decltype(ev)::value><<<grid_of(d.n * d.outs.blocks * d.outs.slabs), 256, 0, st>>>(
                d, static_cast<const T*>(x), weight, bias, static_cast<const T*>(gate),
                reinterpret_cast<const float2*>(stats), static_cast<T*>(y));
            return hipGetLastError();
        });
    });
}

hipError_t launch_group_norm_rows_bwd(const GroupShape& d, const void* dy, const void* x, const float* weight,
                                      const float* bias, const void* gate, const float* stats, void* d_x,
                                      void* d_gate, float* part, hipStream_t st) {
    return by_io(d, [&](auto io_) {
        using IO = decltype(io_);
        using T = typename IO::T;
        return by_vector<IO>(d, [&](auto ev) {
            constexpr int EV = decltype(ev)::value;
            return by_team(d.cg / EV, [&](auto nv, auto ts) {
                constexpr int NV = decltype(nv)::value, TS = decltype(ts)::value;
                k_group_norm_rows_bwd<IO, EV, NV, TS><<<static_cast<unsigned>(d.sums.blocks * d.sums.slabs), 256, 0, st>>>(
                    d, static_cast<const T*>(dy), static_cast<const T*>(x), weight, bias, static_cast<const T*>(gate),
                    stats, static_cast<T*>(d_x), static_cast<T*>(d_gate), part);
                return hipGetLastError();
            });
        });
    });
}

hipError_t launch_group_norm_sums(const GroupShape& d, const void* dy, const void* x, const float* weight,
                                  const float* bias, const void* gate, const float* stats, float* part,
                                  hipStream_t st) {
    return by_io(d, [&](auto io_) {
        using IO = decltype(io_);
        using T = typename IO::T;
        return by_vector<IO>(d, [&](auto ev) {
            k_group_norm_sums<IO, decltype(ev)::value><<<grid_of(d.n * d.sums.blocks * d.sums.slabs), 256, 0, st>>>(
                d, static_cast<const T*>(dy), static_cast<const T*>(x), weight, bias, static_cast<const T*>(gate),
                stats, part);
            return hipGetLastError();
        });
    });
}

hipError_t launch_group_norm_means(const GroupShape& d, const float* part, const float* weight, float* chan,
                                   float* mean, hipStream_t st) {
    k_group_norm_means<<<grid_of(d.n * d.groups), 256, 0, st>>>(d, part, weight, chan, reinterpret_cast<float2*>(mean));
    return hipGetLastError();
}

hipError_t launch_group_norm_grad(const GroupShape& d, const void* dy, const void* x, const float* weight,
                                  const float* bias, const void* gate, const float* stats, const float* mean,
                                  void* d_x, void* d_gate, const float* chan, float* d_weight, float* d_bias,
                                  hipStream_t st) {
    const int sums = d_weight || d_bias ? 2 * ((d.c + 31) / 32) : 0;
    return by_io(d, [&](auto io_) {
        using IO = decltype(io_);
        using T = typename IO::T;
        return by_vector<IO>(d, [&](auto ev) {
            k_group_norm_grad<IO, decltype(ev)::value><<<sums + grid_of(d.n * d.outs.blocks * d.outs.slabs), 256, 0, st>>>(
                d, static_cast<const T*>(dy), static_cast<const T*>(x), weight, bias, static_cast<const T*>(gate),
                stats, reinterpret_cast<const float2*>(mean), static_cast<T*>(d_x), static_cast<T*>(d_gate), chan, sums,
                d_weight, d_bias);
            return hipGetLastError();
        });
    });
}

hipError_t launch_group_norm_weight(const GroupShape& d, const float* part, int64_t parts, float* d_weight,
                                    float* d_bias, hipStream_t st) {
    k_group_norm_weight<<<dim3((d.c + 31) / 32, 2), 1024, 0, st>>>(part, parts, d.c, d_weight, d_bias);
    return hipGetLastError();
}

}  // namespace ssd
