// Linear attention with a constant decay per head, one token from cached states (decoding).
//
// Per (batch row, head) with the state S [p, r] of the row's slot and a = exp(log_decay):
//   S' = a S + v k^T,   y = scale S' q = scale (a (S q) + v (k.q)).
// The dot product is taken of the old state, so that a state element is read once and written once:
// 8 bytes for 5 flops, bound by HBM (64 rows of 80 heads, p = 64, r = 128, bf16 60 us, 5.4 TB/s).  A state row
// (r / 4 float4s) is held by r / 4 consecutive lanes, which add up S q; a thread's state loads are all issued before
// their first use.  The state is updated in place: each element is read and written by the same thread.
#include <type_traits>

#include "delta_device.hpp"
#include "linear_power.hpp"
#include "ssd_launch.hpp"

namespace ssd {

namespace {

__device__ __forceinline__ float dot4(v4f a, v4f b) { return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3]; }

}  // namespace

// R4 = dstate / 4 lanes per state row, P = headdim; a workgroup per (b, h).
template <class IO, int R4, int P>
__global__ __launch_bounds__(NT) void k_linear_step(DeltaShape d, int nslots, const typename IO::T* __restrict__ q,
                                                    const typename IO::T* __restrict__ k,
                                                    const typename IO::T* __restrict__ v,
                                                    const float* __restrict__ log_decay, float* __restrict__ state,
                                                    const int32_t* __restrict__ slots,
                                                    typename IO::T* __restrict__ y) {
    constexpr int ROWS = NT / R4, K = P > ROWS ? P / ROWS : 1;  // rows of a pass, passes
    const int64_t bh = blockIdx.x;
    const int h = static_cast<int>(bh % d.H), b = static_cast<int>(bh / d.H);
    const int c4 = threadIdx.x % R4, row0 = threadIdx.x / R4;
    const int slot = slots ? slots[b] : b;
    if (slot < 0 || slot >= nslots) {  // an idle row
#pragma unroll
        for (int m = 0; m < K; ++m)
            if (c4 == 0 && row0 + m * ROWS < P) io<IO>::st(y, bh * P + row0 + m * ROWS, 0.0f);
        return;
    }
    const int hk = h / (d.H / d.HK);
    v4f* S = reinterpret_cast<v4f*>(state) + (static_cast<int64_t>(slot) * d.H + h) * P * R4;
    v4f s[K];
    float vv[K];
#pragma unroll
    for (int m = 0; m < K; ++m) {
        const int p = row0 + m * ROWS;
        if (p < P) {
            s[m] = __builtin_nontemporal_load(S + p * R4 + c4);
            vv[m] = io<IO>::ld(v, b * d.vs[0] + h * d.vs[2] + p);
        }
    }
    const v4f k4 = io<IO>::ld4(k, b * d.ks[0] + hk * d.ks[2] + 4 * c4);
    const v4f q4 = io<IO>::ld4(q, b * d.qs[0] + hk * d.qs[2] + 4 * c4);
    const float a = power(log2_decay(log_decay[h]), 1);
    const float kq = sum_over_lanes<R4>(dot4(k4, q4));
#pragma unroll
    for (int m = 0; m < K; ++m) {
        const int p = row0 + m * ROWS;
        if (p < P) {  // whole rows are in or out together
            const float sq = sum_over_lanes<R4>(dot4(s[m], q4));
            __builtin_nontemporal_store(a * s[m] + vv[m] * k4, S + p * R4 + c4);
            if (c4 == 0) io<IO>::st(y, bh * P + p, d.scale * (a * sq + vv[m] * kq));
        }
    }
}

namespace {

template <class IO, int R4>
hipError_t step_r(const DeltaShape& d, int nslots, const void* q, const void* k, const void* v,
                  const float* log_decay, float* state, const int32_t* slots, void* y, hipStream_t st) {
    using T = typename IO::T;
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(d.B) * d.H));
    auto run = [&](auto p) {
        k_linear_step<IO, R4, decltype(p)::value>
            <<<grid, NT, 0, st>>>(d, nslots, static_cast<const T*>(q), static_cast<const T*>(k),
                                  static_cast<const T*>(v), log_decay, state, slots, static_cast<T*>(y));
        return hipGetLastError();
    };
    switch (d.P) {
        case 16: return run(std::integral_constant<int, 16>{});
        case 32: return run(std::integral_constant<int, 32>{});
        case 64: return run(std::integral_constant<int, 64>{});
        case 128: return run(std::integral_constant<int, 128>{});
        default: return hipErrorInvalidValue;
    }
}

template <class IO>
hipError_t step_io(const DeltaShape& d, int nslots, const void* q, const void* k, const void* v,
                   const float* log_decay, float* state, const int32_t* slots, void* y, hipStream_t st) {
    switch (d.R) {
        case 16: return step_r<IO, 4>(d, nslots, q, k, v, log_decay, state, slots, y, st);
        case 32: return step_r<IO, 8>(d, nslots, q, k, v, log_decay, state, slots, y, st);
        case 64: return step_r<IO, 16>(d, nslots, q, k, v, log_decay, state, slots, y, st);
        case 128: return step_r<IO, 32>(d, nslots, q, k, v, log_decay, state, slots, y, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_linear_step(const DeltaShape& d, int nslots, const void* q, const void* k, const void* v,
                              const float* log_decay, float* state, const int32_t* slots, void* y, hipStream_t st) {
    return d.io == 1 ? step_io<BF16>(d, nslots, q, k, v, log_decay, state, slots, y, st)
                     : step_io<F32>(d, nslots, q, k, v, log_decay, state, slots, y, st);
}

}  // namespace ssd
