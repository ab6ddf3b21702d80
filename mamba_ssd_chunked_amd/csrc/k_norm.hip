// Root-mean-square norm over rows, with the residual's addition and an 8-bit output.
//
//   s = x + residual,  y = s rsqrt(mean(s^2) + eps) w;
//   8 bits: scale = max|y| / 448 over a row or a group of it (1 where y is all zero),
//           y8 = y / scale rounded to e4m3 (4 exponent, 3 fraction bits, largest value 448).
// Gradient: with rstd = rsqrt(mean(s^2) + eps) and n = s rstd,
//   d_x = d_s + rstd (w dy - n mean(n w dy)),   d_w = sum over rows of dy n.
// A row is read once and kept in registers (the gradient's of more than 16384 values, or of more than
// 8192 that are not whole vectors, partly in scratch: 92 to 376 bytes a thread): bound by HBM.  8192
// rows of 5120 bf16 values with residual, s and 8-bit output: 60 us, 4.9 TB/s; 8192 rows of 1536 in
// fp32: forward 36 us, 5.5 TB/s, gradient 35 us and 5 us for joining the weight gradient; 64 rows: 6 us,
// a launch's latency.  A team of 64, 256 or 1024 threads has a row; a thread's vectors lie a team apart,
// so each load of a team is contiguous.  Sums are fp32; y is rounded once to the io type, and its fp32
// values, not those, are divided for the 8 bits.
// The weight gradient is summed per team over its rows in registers, written once per team, and
// added up by a second kernel in team order: no atomics, bitwise reproducible.
#include <type_traits>

#include "ssd_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {

namespace {

constexpr float kF8Max = 448.0f;

template <class IO, int EV>
__device__ __forceinline__ void ldv(const typename IO::T* p, float (&x)[EV]) {
    if constexpr (EV == 1) {
        x[0] = io<IO>::ld(p, 0);
    } else {
#pragma unroll
        for (int e = 0; e < EV; e += 4) {
            const v4f t = io<IO>::ld4(p, e);
#pragma unroll
            for (int m = 0; m < 4; ++m) x[e + m] = t[m];
        }
    }
}
// bf16 vectors of eight are one 16-byte access
template <>
__device__ __forceinline__ void ldv<BF16, 8>(const uint16_t* p, float (&x)[8]) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(u[e] << 16);
        x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
}
template <class IO, int EV>
__device__ __forceinline__ void stv(typename IO::T* p, const float (&x)[EV]) {
    if constexpr (EV == 1) {
        io<IO>::st(p, 0, x[0]);
    } else if constexpr (EV == 8) {
        uint4 w;
        w.x = f32x2_to_bf16x2(x[0], x[1]);
        w.y = f32x2_to_bf16x2(x[2], x[3]);
        w.z = f32x2_to_bf16x2(x[4], x[5]);
        w.w = f32x2_to_bf16x2(x[6], x[7]);
        *reinterpret_cast<uint4*>(p) = w;
    } else {
        io<IO>::st4(p, 0, v4f{x[0], x[1], x[2], x[3]});
    }
}
template <int EV>
__device__ __forceinline__ void stv8(uint8_t* p, const float (&x)[EV]) {
    if constexpr (EV == 1) {
        p[0] = static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x[0], 0.0f, 0, false) & 0xff);
    } else {
#pragma unroll
        for (int e = 0; e < EV; e += 4) {
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[e], x[e + 1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(x[e + 2], x[e + 3], w, true);
            *reinterpret_cast<int*>(p + e) = w;
        }
    }
}

struct Sum {
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct Max {
    static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};

// Reduce over the threads of a team; all of them get the result.  sh: 16 floats per team, free
// again after the next barrier.
template <int TS, class OP>
__device__ __forceinline__ float team_reduce(float v, float* sh) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = OP::of(v, __shfl_xor(v, o));
    if constexpr (TS > 64) {
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
        __syncthreads();
        v = sh[0];
#pragma unroll
        for (int w = 1; w < TS / 64; ++w) v = OP::of(v, sh[w]);
    }
    return v;
}

constexpr int team_block(int TS) { return TS < 256 ? 256 : TS; }

}  // namespace

// EV values per access, NV accesses per thread, teams of TS threads.
template <class IO, int EV, int NV, int TS>
__global__ __launch_bounds__(team_block(TS)) void k_rms_norm(NormShape n, const typename IO::T* __restrict__ x,
                                                             const typename IO::T* residual,
                                                             const float* __restrict__ weight, typename IO::T* s_out,
                                                             typename IO::T* __restrict__ y, uint8_t* __restrict__ y8,
                                                             float* __restrict__ scale) {
    constexpr int TEAMS = team_block(TS) / TS;
    __shared__ float sh[2][16];
    const int tid = threadIdx.x % TS;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TS;
    if (row >= n.rows) return;  // a whole team; teams smaller than the workgroup share no barrier
    const int64_t at = row * n.width;
    float v[NV][EV], wt[NV][EV];
    float sq = 0.0f;
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int col = (tid + m * TS) * EV;
        if (col < n.width) {
            ldv<IO, EV>(x + at + col, v[m]);
            if (residual) {
                float r[EV];
                ldv<IO, EV>(residual + at + col, r);
#pragma unroll
                for (int e = 0; e < EV; ++e) v[m][e] += r[e];
            }
            ldv<F32, EV < 4 ? EV : 4>(weight + col, *reinterpret_cast<float(*)[EV < 4 ? EV : 4]>(wt[m]));
            if constexpr (EV == 8) ldv<F32, 4>(weight + col + 4, *reinterpret_cast<float(*)[4]>(wt[m] + 4));
        } else {
#pragma unroll
            for (int e = 0; e < EV; ++e) v[m][e] = wt[m][e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < EV; ++e) sq += v[m][e] * v[m][e];
    }
    if (s_out) {
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int col = (tid + m * TS) * EV;
            if (col < n.width) stv<IO, EV>(s_out + at + col, v[m]);
        }
    }
    sq = team_reduce<TS, Sum>(sq, sh[0]);
    const float rstd = 1.0f / sqrtf(sq / static_cast<float>(n.width) + n.eps);
    float top = 0.0f;
#pragma unroll
    for (int m = 0; m < NV; ++m)
#pragma unroll
        for (int e = 0; e < EV; ++e) {
            v[m][e] *= rstd * wt[m][e];
            top = fmaxf(top, fabsf(v[m][e]));
        }
    if (y) {
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int col = (tid + m * TS) * EV;
            if (col < n.width) stv<IO, EV>(y + at + col, v[m]);
        }
    }
    if (!y8) return;
    const bool whole = n.group == n.width;
    if (whole) top = team_reduce<TS, Max>(top, sh[1]);
    const int groups = n.width / n.group;
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int col = (tid + m * TS) * EV;
        if (!whole) {  // a power of two of consecutive lanes holds a group
            top = 0.0f;
#pragma unroll
            for (int e = 0; e < EV; ++e) top = fmaxf(top, fabsf(v[m][e]));
            for (int o = 1; o < n.group / EV; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
        }
        const float sc = top > 0.0f ? top / kF8Max : 1.0f;
        const float up = top < 0x1p-100f ? 0x1p100f : 1.0f;  // below 2^-117 the scale is denormal: fewer bits
        const float by = top > 0.0f ? top * up / kF8Max : 1.0f;
        if (col < n.width) {
            float o[EV];
#pragma unroll
            for (int e = 0; e < EV; ++e) o[e] = v[m][e] * up / by;
            stv8<EV>(y8 + at + col, o);
            if (col % n.group == 0) scale[row * groups + col / n.group] = sc;
        }
    }
}

template <class IO, int EV, int NV, int TS>
__global__ __launch_bounds__(team_block(TS)) void k_rms_norm_bwd(NormShape n, int64_t teams,
                                                                 const typename IO::T* __restrict__ dy,
                                                                 const typename IO::T* __restrict__ s,
                                                                 const typename IO::T* d_s,
                                                                 const float* __restrict__ weight,
                                                                 typename IO::T* d_x, float* __restrict__ part) {
    constexpr int TEAMS = team_block(TS) / TS, EW = EV < 4 ? EV : 4;
    __shared__ float sh[4][16];
    const int tid = threadIdx.x % TS;
    const int64_t team = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TS;
    if (team >= teams) return;  // a whole team, as in the forward
    float wt[NV][EV], dw[NV][EV];
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int col = (tid + m * TS) * EV;
#pragma unroll
        for (int e = 0; e < EV; ++e) wt[m][e] = dw[m][e] = 0.0f;
        if (col < n.width) {
            ldv<F32, EW>(weight + col, *reinterpret_cast<float(*)[EW]>(wt[m]));
            if constexpr (EV == 8) ldv<F32, 4>(weight + col + 4, *reinterpret_cast<float(*)[4]>(wt[m] + 4));
        }
    }
    int flip = 0;
    for (int64_t row = team; row < n.rows; row += teams, flip ^= 2) {
        const int64_t at = row * n.width;
        float v[NV][EV], g[NV][EV];
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int col = (tid + m * TS) * EV;
            if (col < n.width) {
                ldv<IO, EV>(s + at + col, v[m]);
                ldv<IO, EV>(dy + at + col, g[m]);
            } else {
#pragma unroll
                for (int e = 0; e < EV; ++e) v[m][e] = g[m][e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < EV; ++e) {
                sq += v[m][e] * v[m][e];
                dot += v[m][e] * (wt[m][e] * g[m][e]);
            }
        }
        sq = team_reduce<TS, Sum>(sq, sh[flip]);
        dot = team_reduce<TS, Sum>(dot, sh[flip + 1]);
        const float inv_n = 1.0f / static_cast<float>(n.width);
        const float rstd = 1.0f / sqrtf(sq * inv_n + n.eps);
        const float c = dot * inv_n * rstd * rstd;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int col = (tid + m * TS) * EV;
            float o[EV];
#pragma unroll
            for (int e = 0; e < EV; ++e) {
                o[e] = rstd * (wt[m][e] * g[m][e] - v[m][e] * c);
                dw[m][e] += g[m][e] * (v[m][e] * rstd);
            }
            if (col < n.width) {
                if (d_s) {
                    float r[EV];
                    ldv<IO, EV>(d_s + at + col, r);
#pragma unroll
                    for (int e = 0; e < EV; ++e) o[e] += r[e];
                }
                stv<IO, EV>(d_x + at + col, o);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int col = (tid + m * TS) * EV;
        if (col < n.width) {
            float* p = part + team * n.width + col;
            if constexpr (EV == 1) p[0] = dw[m][0];
            else {
#pragma unroll
                for (int e = 0; e < EV; e += 4)
                    *reinterpret_cast<v4f*>(p + e) = v4f{dw[m][e], dw[m][e + 1], dw[m][e + 2], dw[m][e + 3]};
            }
        }
    }
}

// d_weight[col] = sum of the teams' partial sums: 32 columns x 32 interleaved runs of teams.
__global__ __launch_bounds__(1024) void k_rms_norm_weight(const float* __restrict__ part, int64_t teams, int width,
                                                          float* __restrict__ d_weight) {
    __shared__ float sh[32][33];
    const int c = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int col = static_cast<int>(blockIdx.x) * 32 + c;
    float acc = 0.0f;
    if (col < width) {
#pragma unroll 8  // as many loads under way
        for (int64_t t = run; t < teams; t += 32) acc += part[t * width + col];
    }
    sh[run][c] = acc;
    __syncthreads();
    if (run == 0 && col < width) {
        acc = 0.0f;
#pragma unroll
        for (int m = 0; m < 32; ++m) acc += sh[m][c];
        d_weight[col] = acc;
    }
}

namespace {

// Calls f with the access width, accesses per thread and team size for rows of `width`: the
// smallest team whose threads hold at most four 16-byte vectors of a row (eight where even 1024
// threads need more); single values where rows are not whole vectors.
template <class IO, class F>
hipError_t by_width(int width, F&& f) {
    constexpr int V = 16 / sizeof(typename IO::T);
    auto vec = [&](auto ts) {
        constexpr int TS = decltype(ts)::value;
        const int nv = (width / V + TS - 1) / TS;
        if constexpr (TS == 64)
            if (nv <= 1) return f(std::integral_constant<int, V>{}, std::integral_constant<int, 1>{}, ts);
        if (nv <= 2) return f(std::integral_constant<int, V>{}, std::integral_constant<int, 2>{}, ts);
        if (nv <= 3) return f(std::integral_constant<int, V>{}, std::integral_constant<int, 3>{}, ts);
        if (nv <= 4) return f(std::integral_constant<int, V>{}, std::integral_constant<int, 4>{}, ts);
        if constexpr (TS == 1024 && V == 4)  // bf16 rows of the widest width have four
            if (nv <= 8) return f(std::integral_constant<int, V>{}, std::integral_constant<int, 8>{}, ts);
        return hipErrorInvalidValue;
    };
    if (width % V == 0) {
        if (width <= 4 * 64 * V) return vec(std::integral_constant<int, 64>{});
        if (width <= 4 * 256 * V) return vec(std::integral_constant<int, 256>{});
        return vec(std::integral_constant<int, 1024>{});
    }
    const std::integral_constant<int, 1> one;
    if (width <= 4 * 64) return f(one, std::integral_constant<int, 4>{}, std::integral_constant<int, 64>{});
    if (width <= 4 * 256) return f(one, std::integral_constant<int, 4>{}, std::integral_constant<int, 256>{});
    if (width <= 8 * 1024) return f(one, std::integral_constant<int, 8>{}, std::integral_constant<int, 1024>{});
    return f(one, std::integral_constant<int, 32>{}, std::integral_constant<int, 1024>{});
}

template <class IO>
hipError_t norm_io(const NormShape& n, const void* x, const void* residual, const float* weight, void* s, void* y,
                   void* y8, float* scale, hipStream_t st) {
    using T = typename IO::T;
    return by_width<IO>(n.width, [&](auto ev, auto nv, auto ts) {
        constexpr int EV = decltype(ev)::value, NV = decltype(nv)::value, TS = decltype(ts)::value;
        constexpr int BLK = team_block(TS), TEAMS = BLK / TS;
        const dim3 grid(static_cast<unsigned>((n.rows + TEAMS - 1) / TEAMS));
        k_rms_norm<IO, EV, NV, TS><<<grid, BLK, 0, st>>>(n, static_cast<const T*>(x), static_cast<const T*>(residual),
                                                        weight, static_cast<T*>(s), static_cast<T*>(y),
                                                        static_cast<uint8_t*>(y8), scale);
        return hipGetLastError();
    });
}

template <class IO>
hipError_t norm_bwd_io(const NormShape& n, const void* dy, const void* s, const void* d_s, const float* weight,
                       void* d_x, float* part, hipStream_t st) {
    using T = typename IO::T;
    const int64_t teams = rms_norm_parts(n.rows);
    return by_width<IO>(n.width, [&](auto ev, auto nv, auto ts) {
        constexpr int EV = decltype(ev)::value, NV = decltype(nv)::value, TS = decltype(ts)::value;
        constexpr int BLK = team_block(TS), TEAMS = BLK / TS;
        const dim3 grid(static_cast<unsigned>((teams + TEAMS - 1) / TEAMS));
        k_rms_norm_bwd<IO, EV, NV, TS><<<grid, BLK, 0, st>>>(n, teams, static_cast<const T*>(dy),
                                                            static_cast<const T*>(s), static_cast<const T*>(d_s),
                                                            weight, static_cast<T*>(d_x), part);
        return hipGetLastError();
    });
}

}  // namespace

int64_t rms_norm_parts(int64_t rows) { return rows < 1024 ? rows : 1024; }

hipError_t launch_rms_norm(const NormShape& n, const void* x, const void* residual, const float* weight, void* s,
                           void* y, void* y8, float* scale, hipStream_t st) {
    return n.io == 1 ? norm_io<BF16>(n, x, residual, weight, s, y, y8, scale, st)
                     : norm_io<F32>(n, x, residual, weight, s, y, y8, scale, st);
}

hipError_t launch_rms_norm_bwd(const NormShape& n, const void* dy, const void* s, const void* d_s,
                               const float* weight, void* d_x, float* part, hipStream_t st) {
    return n.io == 1 ? norm_bwd_io<BF16>(n, dy, s, d_s, weight, d_x, part, st)
                     : norm_bwd_io<F32>(n, dy, s, d_s, weight, d_x, part, st);
}

hipError_t launch_rms_norm_weight(const NormShape& n, const float* part, float* d_weight, hipStream_t st) {
    k_rms_norm_weight<<<dim3(static_cast<unsigned>((n.width + 31) / 32)), 1024, 0, st>>>(part, rms_norm_parts(n.rows),
                                                                                        n.width, d_weight);
    return hipGetLastError();
}

}  // namespace ssd
