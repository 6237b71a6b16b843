// la_step.cuh -- one decode token of the decay linear attention:
//     S <- e^g S + k v^T;   o = scale S^T q
// for B x H independent D x D fp32 states, read once and written once (in place or to
// another buffer).
//
// 8 D^2 bytes of state for 5 D^2 operations: bound by HBM while many states are in
// flight (1024 x 32 states of 64: 162 us, 6.73 TB/s, 1.03 of a plain copy's rate), and by the
// latency of one state's round trip for a few.  A block owns 64
// columns of one state; lane l of a warp holds columns 4 (l % 16) .. +3 of rows of half
// l / 16, so a warp's load covers two 256-byte row pieces.  Two splits of the D rows over
// warps: 64 rows a warp (32 float4 in flight per lane) where the states fill the GPU, and 16
// warps' worth of shorter columns (8 to 16 rows a warp) for a few states, where every
// load of a state then leaves at once and the sums add one barrier.
#pragma once
#include "common.cuh"
#include "la_common.cuh"

namespace wkv7 {
namespace la {

// W warps share the D rows; kUnits states per block.
template <typename Tin, int D, int W, int kUnits>
__global__ void __launch_bounds__(32 * W * kUnits)
la_step_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
               const Tin* __restrict__ g, int g_per_head, const float* state, float* out_state,
               Tin* __restrict__ o, long long units, int H, float scale) {
    constexpr int R = D / (2 * W);  // rows per lane
    constexpr int kSlabs = D / 64;
    __shared__ __align__(16) float sum[W > 1 ? W : 1][kUnits][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = warp / W, w = warp % W;
    const long long id = (long long)blockIdx.x * kUnits + sub;
    const long long unit = id / kSlabs;
    const int slab = (int)(id - unit * kSlabs);
    const bool live = unit < units;  // warp-uniform
    const int c = lane & 15, row0 = w * 2 * R + (lane >> 4) * R;
    float4 S[R];
    const long long at = live ? unit * D * D + 64 * slab + 4 * c : 0;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            S[i] = *reinterpret_cast<const float4*>(state + at + (long long)(row0 + i) * D);
        const float d = expf(to_f32(g[g_per_head ? unit % H : unit]));
        const float4 vv = load4(v + unit * D + 64 * slab + 4 * c);
#pragma unroll
        for (int i = 0; i < R; i += 4) {
            const float4 k4 = load4(k + unit * D + row0 + i), q4 = load4(q + unit * D + row0 + i);
            const float kv[4] = {k4.x, k4.y, k4.z, k4.w}, qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float4& s = S[i + r];
                s.x = fmaf(d, s.x, kv[r] * vv.x);
                s.y = fmaf(d, s.y, kv[r] * vv.y);
                s.z = fmaf(d, s.z, kv[r] * vv.z);
                s.w = fmaf(d, s.w, kv[r] * vv.w);
                acc.x = fmaf(s.x, qv[r], acc.x);
                acc.y = fmaf(s.y, qv[r], acc.y);
                acc.z = fmaf(s.z, qv[r], acc.z);
                acc.w = fmaf(s.w, qv[r], acc.w);
                *reinterpret_cast<float4*>(out_state + at + (long long)(row0 + i + r) * D) = s;
            }
        }
    }
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
    if (W > 1) {
        if (lane < 16) *reinterpret_cast<float4*>(&sum[w][sub][4 * c]) = acc;
        __syncthreads();
        if (w != 0 || lane >= 16) return;
#pragma unroll
        for (int i = 1; i < W; ++i) {
            const float4 s = *reinterpret_cast<const float4*>(&sum[i][sub][4 * c]);
            acc.x += s.x;
            acc.y += s.y;
            acc.z += s.z;
            acc.w += s.w;
        }
    }
    if (live && lane < 16)
        store4(o + unit * D + 64 * slab + 4 * c,
               make_float4(scale * acc.x, scale * acc.y, scale * acc.z, scale * acc.w));
}

template <typename Tin, int D>
inline cudaError_t launch_la_step_d(const Tin* q, const Tin* k, const Tin* v, const Tin* g,
                                    int g_per_head, const float* state, float* out_state, Tin* o,
                                    long long units, int H, float scale, cudaStream_t stream) {
    constexpr int kSlabs = D / 64, kBig = D / 64, kSmall = D == 256 ? 16 : D / 8;
    // The fine split up to 592 blocks, the wide one above it (as many bytes in flight, fewer
    // barriers).  Fine and wide, us a call: 32 states of 64, 1.7 and 2.8; 32 of 128, 2.1 and
    // 2.7; 576 of 64, 3.2 and 3.3; 1184 of 64, 5.1 and 5.2; 1184 of 128, 16.7 and 15.6.
    if (units * kSlabs <= 148 * 4) {
        la_step_kernel<Tin, D, kSmall, 1><<<(unsigned)(units * kSlabs), 32 * kSmall, 0, stream>>>(
            q, k, v, g, g_per_head, state, out_state, o, units, H, scale);
    } else {
        constexpr int kUnits = 4 / kBig;
        const long long blocks = (units * kSlabs + kUnits - 1) / kUnits;
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        la_step_kernel<Tin, D, kBig, kUnits><<<(unsigned)blocks, 32 * kBig * kUnits, 0, stream>>>(
            q, k, v, g, g_per_head, state, out_state, o, units, H, scale);
    }
    return cudaGetLastError();
}

template <typename Tin>
inline cudaError_t launch_la_step(const void* q, const void* k, const void* v, const void* g,
                                  int g_per_head, const float* state, float* out_state, void* o,
                                  long long units, int H, int D, float scale,
                                  cudaStream_t stream) {
    const Tin *q_ = static_cast<const Tin*>(q), *k_ = static_cast<const Tin*>(k),
              *v_ = static_cast<const Tin*>(v), *g_ = static_cast<const Tin*>(g);
    Tin* o_ = static_cast<Tin*>(o);
    return D == 64    ? launch_la_step_d<Tin, 64>(q_, k_, v_, g_, g_per_head, state, out_state, o_,
                                                  units, H, scale, stream)
           : D == 128 ? launch_la_step_d<Tin, 128>(q_, k_, v_, g_, g_per_head, state, out_state,
                                                   o_, units, H, scale, stream)
                      : launch_la_step_d<Tin, 256>(q_, k_, v_, g_, g_per_head, state, out_state,
                                                   o_, units, H, scale, stream);
}

}  // namespace la
}  // namespace wkv7
