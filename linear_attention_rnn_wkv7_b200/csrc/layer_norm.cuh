// layer_norm.cuh -- layer norm of rows of D elements, forward and backward:
//     mean = sum x / D, rstd = (sum (x - mean)^2 / D + eps)^-1/2, xh = (x - mean) rstd
//     y  = xh w + b
//     dx = rstd (u - sum u / D - xh sum(u xh) / D),  u = dy w
//     dw = sum over rows dy xh,  db = sum over rows dy
// Rows come in G groups with a weight and bias each (one group: layer norm; a group per
// head: the norm of a mixing layer's output): row r is of group (r / inner) % G, inner = 1
// for [.., G, D] rows and T for head-first [B, G, T, D] ones.
//
// Bound by HBM: x once in and y once out (x, dy in, dx out).  A team of threads holds a row
// in registers, while the next one's loads are already in flight.  Statistics take one
// exchange: each thread has the mean and the sum of squares around it of its own
// elements, and pairs merge as (n, m, M2): m += d n2 / n12, M2 += M2' + d^2 n1 n2 / n12 with d
// the means' difference (no cancellation of two large sums, no second read).  Team t works on
// rows of group t % G only: w and b stay in registers over its rows, and in the backward so do
// its sums of dw and db, written once at the end; a second kernel adds the teams' sums in a
// fixed order (no atomics: the result does not depend on scheduling).  Consecutive teams
// hold consecutive groups, so a block's loads are contiguous for every layout with inner = 1.
//
// All statistics and sums are fp32.  Above 8192 elements the backward's registers no longer
// hold a row and its sums of dw and db, so those get a kernel of their own, which reads x
// and dy again by columns.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"

namespace wkv7 {
namespace ln {

struct Shape {
    long long rows, inner;
    int G, D;
    long long teams;    // teams in all; team t: group t % G, rows t / G, t / G + S, ..
    float eps;
};
// The k-th row of a group.
__device__ __forceinline__ long long row_at(const Shape& s, long long k, int group) {
    if (s.inner == 1) return k * s.G + group;
    const long long b = k / s.inner;
    return (b * s.G + group) * s.inner + (k - b * s.inner);
}

// VEC consecutive elements as fp32.
template <int VEC> __device__ __forceinline__ void load(const float* p, float (&v)[VEC]) {
    if constexpr (VEC == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = p[i];
    }
}
template <int VEC> __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        const uint32_t r[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __bfloat162float(p[i]);
    }
}
template <int VEC> __device__ __forceinline__ void store(float* p, const float (&v)[VEC]) {
    if constexpr (VEC == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = v[i];
    }
}
template <int VEC> __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = __float2bfloat16_rn(v[i]);
    }
}

// Pairs of fp32 in one instruction: per element the arithmetic of a row is then half, and HBM
// and not the issue rate bounds the kernels (forward of 32768 x 4096 bf16: 193 us without).
__device__ __forceinline__ float sum2(uint64_t x) {
    float a, b;
    split2(x, a, b);
    return a + b;
}
using wkv7::add2;
using wkv7::fma2;
using wkv7::mul2;
// A lone value (rows of odd lengths) goes through the same code.
__device__ __forceinline__ float sum2(float x) { return x; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
template <int VEC> struct PairOf { typedef uint64_t type; };
template <> struct PairOf<1> { typedef float type; };
template <int VEC> using Pair = typename PairOf<VEC>::type;
template <int VEC> constexpr int pairs() { return VEC == 1 ? 1 : VEC / 2; }
template <int VEC> __device__ __forceinline__ Pair<VEC> splat(float x) {
    if constexpr (VEC == 1) return x;
    else return pair2(x, x);
}
template <int VEC> __device__ __forceinline__ void to_pairs(const float (&v)[VEC], Pair<VEC> (&p)[pairs<VEC>()]) {
    if constexpr (VEC == 1) {
        p[0] = v[0];
    } else {
#pragma unroll
        for (int q = 0; q < VEC / 2; ++q) p[q] = pair2(v[2 * q], v[2 * q + 1]);
    }
}
template <int VEC> __device__ __forceinline__ void from_pairs(const Pair<VEC> (&p)[pairs<VEC>()], float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = p[0];
    } else {
#pragma unroll
        for (int q = 0; q < VEC / 2; ++q) split2(p[q], v[2 * q], v[2 * q + 1]);
    }
}

// VEC elements as they are in memory (prefetched rows), and as fp32.
template <typename T, int VEC> struct Raw { T v[VEC]; };
template <> struct Raw<__nv_bfloat16, 8> { uint4 v; };
template <> struct Raw<float, 8> { float4 v[2]; };
template <> struct Raw<float, 4> { float4 v; };
template <typename T, int VEC> __device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
    return *reinterpret_cast<const Raw<T, VEC>*>(p);
}
template <int VEC> __device__ __forceinline__ void unpack(const Raw<float, VEC>& r, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        v[0] = r.v[0].x; v[1] = r.v[0].y; v[2] = r.v[0].z; v[3] = r.v[0].w;
        v[4] = r.v[1].x; v[5] = r.v[1].y; v[6] = r.v[1].z; v[7] = r.v[1].w;
    } else if constexpr (VEC == 4) {
        v[0] = r.v.x; v[1] = r.v.y; v[2] = r.v.z; v[3] = r.v.w;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = r.v[i];
    }
}
template <int VEC>
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, VEC>& r, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __bfloat162float(r.v[i]);
    }
}

// Sums of NS values over a team of TPR threads (a power of two; several teams a block when
// TPR <= 32; above it the block is one team).  Every thread gets the sums.
template <int TPR, int NS>
__device__ __forceinline__ void team_sum(float (&s)[NS], float (*red)[32]) {
    constexpr int kIn = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int m = kIn / 2; m > 0; m >>= 1)
#pragma unroll
        for (int j = 0; j < NS; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], m);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
#pragma unroll
            for (int j = 0; j < NS; ++j) red[j][warp] = s[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            float t = lane < W ? red[j][lane] : 0.f;
#pragma unroll
            for (int m = W / 2; m > 0; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
            s[j] = __shfl_sync(0xffffffffu, t, 0);
        }
    }
}

// Merging (n, mean, M2) over a team: the counts are the same for every row, so each level's
// n2 / n12 and n1 n2 / n12 are made once.
template <int TPR>
struct Merge {
    static constexpr int kIn = TPR < 32 ? TPR : 32, kWarps = TPR / 32;
    static constexpr int levels(int n) { return n <= 1 ? 0 : 1 + levels(n / 2); }
    static constexpr int kA = levels(kIn), kB = levels(kWarps);
    float r[kA + kB + 1], c[kA + kB + 1];

    __device__ __forceinline__ void level(float& n, int l, int m) {
        const float n2 = __shfl_xor_sync(0xffffffffu, n, m), tot = n + n2;
        r[l] = tot > 0.f ? n2 / tot : 0.f;
        c[l] = n * r[l];
        n = tot;
    }
    __device__ __forceinline__ explicit Merge(float n, float* red) {
#pragma unroll
        for (int l = 0; l < kA; ++l) level(n, l, 1 << l);
        if constexpr (TPR > 32) {
            const int lane = threadIdx.x & 31;
            if (lane == 0) red[threadIdx.x >> 5] = n;
            __syncthreads();
            n = lane < kWarps ? red[lane] : 0.f;
#pragma unroll
            for (int l = 0; l < kB; ++l) level(n, kA + l, 1 << l);
            __syncthreads();
        }
    }
    __device__ __forceinline__ void merge(float& mean, float& m2, int l, int m) const {
        const float d = __shfl_xor_sync(0xffffffffu, mean, m) - mean;
        m2 += __shfl_xor_sync(0xffffffffu, m2, m);
        mean = fmaf(d, r[l], mean);
        // (c d first: 0 for a thread without elements, where d, the mean itself, may have a
        // square beyond fp32)
        m2 = fmaf(c[l] * d, d, m2);
    }
    // Mean and sum of squares around it over the team, from each thread's; all get the same.
    __device__ __forceinline__ void operator()(float& mean, float& m2, float (*red)[32]) const {
#pragma unroll
        for (int l = 0; l < kA; ++l) merge(mean, m2, l, 1 << l);
        const int lane = threadIdx.x & 31;
        if constexpr (TPR > 32) {
            const int warp = threadIdx.x >> 5;
            if (lane == 0) {
                red[0][warp] = mean;
                red[1][warp] = m2;
            }
            __syncthreads();
            mean = lane < kWarps ? red[0][lane] : 0.f;
            m2 = lane < kWarps ? red[1][lane] : 0.f;
#pragma unroll
            for (int l = 0; l < kB; ++l) merge(mean, m2, kA + l, 1 << l);
        }
        // (the two lanes of a merge may differ in its last bit)
        mean = __shfl_sync(0xffffffffu, mean, TPR >= 32 ? 0 : lane & ~(TPR - 1));
        m2 = __shfl_sync(0xffffffffu, m2, TPR >= 32 ? 0 : lane & ~(TPR - 1));
    }
};

// Threads of a block.
template <int TPR> constexpr int block_threads() { return TPR <= 32 ? 128 : TPR; }
// Blocks per SM, by the registers that a row of N elements a thread, the next one, the weights and
// (backward) the sums of dw and db take.
template <int TPR, int N> constexpr int fwd_blocks() {
    constexpr int threads = N <= 16 ? 640 : 512;
    return threads / block_threads<TPR>() > 0 ? threads / block_threads<TPR>() : 1;
}
template <int TPR, int N> constexpr int bwd_blocks() {
    constexpr int threads = N <= 8 ? 768 : 512;
    return threads / block_threads<TPR>() > 0 ? threads / block_threads<TPR>() : 1;
}

// A team of TPR threads holds NI groups of VEC elements a thread (groups past D are skipped;
// VEC divides D).
template <typename T, typename Tw, int TPR, int NI, int VEC>
__global__ void __launch_bounds__(block_threads<TPR>(), fwd_blocks<TPR, NI * VEC>())
ln_fwd_kernel(const T* __restrict__ x, const Tw* __restrict__ w, const Tw* __restrict__ b,
              T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd, Shape s) {
    __shared__ float red[2][2][32];
    constexpr int kTeams = block_threads<TPR>() / TPR, P = pairs<VEC>();
    // 1024 threads have 64 registers each: long rows leave none for the weights, which come
    // from L1 each row then (32768 x 4096 bf16 with fp32 weights: held 134 us, not held 177 us).
    constexpr bool kHold = TPR < 1024 || NI * VEC <= 8;
    // Rows on their way: short rows leave registers for three (262144 x 64: 31 us with one, 23
    // with three), longer ones do not (32768 x 4096: 134 us with one, 146 with three)
    constexpr int kDepth = TPR < 1024 && NI * VEC <= 8 ? 3 : 1;
    const int lane = threadIdx.x % TPR;
    const long long team = (long long)blockIdx.x * kTeams + threadIdx.x / TPR;
    const bool in = team < s.teams;
    const int group = in ? (int)(team % s.G) : 0;
    const long long per = s.rows / s.G, step = s.teams / s.G;
    // Every team of a block runs as many turns as its first (whole warps stay together
    // for the shuffles); rows past the end are not loaded or stored.
    const long long first = in ? team / s.G : 0;
    const long long turns = (per - (long long)blockIdx.x * kTeams / s.G + step - 1) / step;
    const long long wo = (long long)group * s.D;
    float count = 0.f;
    Raw<T, VEC> next[kDepth][NI];
    Raw<Tw, VEC> wr[NI], br[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = (i * TPR + lane) * VEC;
        if (e < s.D) {
            count += (float)VEC;
            if (kHold && w) wr[i] = load_raw<Tw, VEC>(w + wo + e);
            if (kHold && b) br[i] = load_raw<Tw, VEC>(b + wo + e);
        }
    }
    auto fetch = [&](long long k, Raw<T, VEC> (&next)[NI]) {
        if (!in || k >= per) return;
        const T* px = x + row_at(s, k, group) * s.D;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (e < s.D) next[i] = load_raw<T, VEC>(px + e);
        }
    };
    const float inv_n = count > 0.f ? 1.f / count : 0.f, inv_d = 1.f / (float)s.D;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) fetch(first + d * step, next[d]);
    const Merge<TPR> merge(count, red[0][0]);
    auto one = [&](long long turn, Raw<T, VEC> (&next)[NI]) {
        const long long k = first + turn * step;
        const bool ok = in && k < per;
        Pair<VEC> xr[NI][P], sum = 0;
        float m, m2;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const bool live = ok && (i * TPR + lane) * VEC < s.D;
            float v[VEC];
            if (live) {
                unpack<VEC>(next[i], v);
            } else {
#pragma unroll
                for (int q = 0; q < VEC; ++q) v[q] = 0.f;
            }
            to_pairs<VEC>(v, xr[i]);
#pragma unroll
            for (int q = 0; q < P; ++q) sum = add2(sum, xr[i][q]);
        }
        fetch(k + kDepth * step, next);
        m = sum2(sum) * inv_n;
        const Pair<VEC> mm = splat<VEC>(-m);
        sum = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if ((i * TPR + lane) * VEC < s.D) {
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const Pair<VEC> d = add2(xr[i][q], mm);
                    sum = fma2(d, d, sum);
                }
            }
        }
        m2 = sum2(sum);
        merge(m, m2, red[turn & 1]);
        const float r = 1.f / sqrtf(m2 * inv_d + s.eps);
        if (ok) {
            const long long row = row_at(s, k, group);
            T* py = y + row * s.D;
            const Pair<VEC> rr = splat<VEC>(r), minus = splat<VEC>(-m);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = (i * TPR + lane) * VEC;
                if (e < s.D) {
                    Pair<VEC> wp[P], bp[P];
                    float v[VEC];
                    if (w) {
                        if (!kHold) wr[i] = load_raw<Tw, VEC>(w + wo + e);
                        unpack<VEC>(wr[i], v);
                        to_pairs<VEC>(v, wp);
                    }
                    if (b) {
                        if (!kHold) br[i] = load_raw<Tw, VEC>(b + wo + e);
                        unpack<VEC>(br[i], v);
                        to_pairs<VEC>(v, bp);
                    }
#pragma unroll
                    for (int q = 0; q < P; ++q) {
                        Pair<VEC> t = mul2(add2(xr[i][q], minus), rr);
                        if (w && b) t = fma2(t, wp[q], bp[q]);
                        else if (w) t = mul2(t, wp[q]);
                        else if (b) t = add2(t, bp[q]);
                        xr[i][q] = t;
                    }
                    from_pairs<VEC>(xr[i], v);
                    store<VEC>(py + e, v);
                }
            }
            if (lane == 0) {
                if (mean) mean[row] = m;
                if (rstd) rstd[row] = r;
            }
        }
    };
    for (long long turn = 0; turn < turns; turn += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            if (turn + d < turns) one(turn + d, next[d]);
    }
}

// part: [S][2][G][D], the sums of dy xh and of dy of S = teams / G teams a group, or with
// kBlockSum (one group, several teams a block) of S = blocks.
template <typename T, typename Tw, int TPR, int NI, int VEC, bool kParam, bool kBlockSum>
__global__ void __launch_bounds__(block_threads<TPR>(), bwd_blocks<TPR, NI * VEC>())
ln_bwd_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ mean,
              const float* __restrict__ rstd, const Tw* __restrict__ w, T* __restrict__ dx,
              float* __restrict__ part, Shape s) {
    __shared__ float red[2][2][32];
    constexpr int kTeams = block_threads<TPR>() / TPR;
    // (1024 threads have 64 registers each: no room for the next row beside a long one)
    constexpr bool kPrefetch = TPR < 1024 || NI * VEC <= 8;
    const int lane = threadIdx.x % TPR;
    const long long team = (long long)blockIdx.x * kTeams + threadIdx.x / TPR;
    const bool in = team < s.teams;
    const int group = in ? (int)(team % s.G) : 0;
    const long long per = s.rows / s.G, step = s.teams / s.G;
    const float inv = 1.f / (float)s.D;
    const long long first = in ? team / s.G : 0;
    const long long turns = (per - (long long)blockIdx.x * kTeams / s.G + step - 1) / step;
    const long long wo = (long long)group * s.D;
    constexpr int P = pairs<VEC>();
    Pair<VEC> dwp[kParam ? NI : 1][P], dbp[kParam ? NI : 1][P];
#pragma unroll
    for (int i = 0; i < (kParam ? NI : 1); ++i)
#pragma unroll
        for (int q = 0; q < P; ++q) dwp[i][q] = dbp[i][q] = 0;
    Raw<Tw, VEC> wr[NI];
    Raw<T, VEC> nx[NI], nd[NI];
    float nm = 0.f, nr = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = (i * TPR + lane) * VEC;
        if (kPrefetch && w && e < s.D) wr[i] = load_raw<Tw, VEC>(w + wo + e);
    }
    auto fetch = [&](long long k) {
        if (!in || k >= per) return;
        const long long row = row_at(s, k, group);
        nm = mean[row];
        nr = rstd[row];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (e < s.D) {
                nx[i] = load_raw<T, VEC>(x + row * s.D + e);
                nd[i] = load_raw<T, VEC>(dy + row * s.D + e);
            }
        }
    };
    if (kPrefetch) fetch(first);
    long long k = first;
    for (long long turn = 0; turn < turns; ++turn, k += step) {
        const bool ok = in && k < per;
        if (!kPrefetch) fetch(k);
        const float m = nm, r = nr;
        Pair<VEC> xh[NI][P], u[NI][P], s0 = 0, s1 = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (ok && (i * TPR + lane) * VEC < s.D) {
                float v[VEC];
                unpack<VEC>(nx[i], v);
                to_pairs<VEC>(v, xh[i]);
                unpack<VEC>(nd[i], v);
                to_pairs<VEC>(v, u[i]);
            }
        }
        if (kPrefetch) fetch(k + step);
        const Pair<VEC> rr = splat<VEC>(r), minus = splat<VEC>(-m);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (ok && (i * TPR + lane) * VEC < s.D) {
                Pair<VEC> wp[P];
                if (w && !kPrefetch) wr[i] = load_raw<Tw, VEC>(w + wo + (i * TPR + lane) * VEC);
                if (w) {
                    float v[VEC];
                    unpack<VEC>(wr[i], v);
                    to_pairs<VEC>(v, wp);
                }
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    xh[i][q] = mul2(add2(xh[i][q], minus), rr);
                    if (kParam) {
                        dwp[i][q] = fma2(u[i][q], xh[i][q], dwp[i][q]);
                        dbp[i][q] = add2(dbp[i][q], u[i][q]);
                    }
                    if (w) u[i][q] = mul2(u[i][q], wp[q]);
                    s0 = add2(s0, u[i][q]);
                    s1 = fma2(u[i][q], xh[i][q], s1);
                }
            }
        }
        float a[2] = {sum2(s0), sum2(s1)};
        team_sum<TPR, 2>(a, red[turn & 1]);
        const Pair<VEC> c0 = splat<VEC>(-a[0] * inv), c1 = splat<VEC>(-a[1] * inv);
        if (ok) {
            T* pd = dx + row_at(s, k, group) * s.D;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = (i * TPR + lane) * VEC;
                if (e < s.D) {
                    float v[VEC];
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        xh[i][q] = mul2(rr, fma2(xh[i][q], c1, add2(u[i][q], c0)));
                    from_pairs<VEC>(xh[i], v);
                    store<VEC>(pd + e, v);
                }
            }
        }
    }
    float dw[kParam ? NI : 1][VEC], db[kParam ? NI : 1][VEC];
#pragma unroll
    for (int i = 0; i < (kParam ? NI : 1); ++i) {
        from_pairs<VEC>(dwp[i], dw[i]);
        from_pairs<VEC>(dbp[i], db[i]);
    }
    if constexpr (kParam && kBlockSum) {
        // the block's teams, in order, through shared memory
        __shared__ float sums[2][kTeams][TPR * NI * VEC];
        const int t = threadIdx.x / TPR;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                sums[0][t][(i * TPR + lane) * VEC + q] = dw[i][q];
                sums[1][t][(i * TPR + lane) * VEC + q] = db[i][q];
            }
        __syncthreads();
        float* p = part + (long long)blockIdx.x * 2 * s.D;
        for (int e = threadIdx.x; e < 2 * s.D; e += block_threads<TPR>()) {
            const int which = e >= s.D, c = which ? e - s.D : e;
            float a = 0.f;
#pragma unroll
            for (int j = 0; j < kTeams; ++j) a += sums[which][j][c];
            p[e] = a;
        }
    } else if (kParam && in) {
        float* p = part + (team / s.G) * 2 * s.G * s.D + wo;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (e < s.D) {
                if constexpr (VEC == 1) {
                    p[e] = dw[i][0];
                    p[(long long)s.G * s.D + e] = db[i][0];
                } else {
#pragma unroll
                    for (int q = 0; q < VEC; q += 4) {
                        *reinterpret_cast<float4*>(p + e + q) =
                            make_float4(dw[i][q], dw[i][q + 1], dw[i][q + 2], dw[i][q + 3]);
                        *reinterpret_cast<float4*>(p + (long long)s.G * s.D + e + q) =
                            make_float4(db[i][q], db[i][q + 1], db[i][q + 2], db[i][q + 3]);
                    }
                }
            }
        }
    }
}

// The same sums by columns: VEC columns a thread, rows blockIdx.y, + S, .. of their group.
template <typename T, int VEC>
__global__ void __launch_bounds__(128)
ln_bwd_cols_kernel(const T* __restrict__ x, const T* __restrict__ dy,
                   const float* __restrict__ mean, const float* __restrict__ rstd,
                   float* __restrict__ part, Shape s) {
    const long long cols = (long long)s.G * s.D;
    const long long c = ((long long)blockIdx.x * 128 + threadIdx.x) * VEC;
    if (c >= cols) return;
    const int group = (int)(c / s.D), e = (int)(c - (long long)group * s.D);
    float dw[VEC], db[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) dw[q] = db[q] = 0.f;
#pragma unroll 4
    for (long long k = blockIdx.y; k < s.rows / s.G; k += gridDim.y) {
        const long long row = row_at(s, k, group);
        const float m = mean[row], r = rstd[row];
        float xv[VEC], dv[VEC];
        load<VEC>(x + row * s.D + e, xv);
        load<VEC>(dy + row * s.D + e, dv);
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            dw[q] = fmaf(dv[q], (xv[q] - m) * r, dw[q]);
            db[q] += dv[q];
        }
    }
    float* p = part + (long long)blockIdx.y * 2 * cols + c;
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
        p[q] = dw[q];
        p[cols + q] = db[q];
    }
}

// dw, db [G D] from part [S][2][G D]: 8 warps share the S partial sums of 32 columns.
template <typename Tw>
__global__ void __launch_bounds__(256)
ln_param_kernel(const float* __restrict__ part, long long S, long long cols, Tw* __restrict__ dw,
                Tw* __restrict__ db) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + lane;  // 2 * cols columns
    float a = 0.f;
    if (c < 2 * cols)
#pragma unroll 8
        for (long long i = warp; i < S; i += 8) a += part[i * 2 * cols + c];
    red[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && c < 2 * cols) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a += red[i][lane];
        if (c < cols) {
            if (dw) dw[c] = from_f32<Tw>(a);
        } else if (db) {
            db[c - cols] = from_f32<Tw>(a);
        }
    }
}

// Threads per row and elements per thread for a row of D: teams of 4 to 32 threads while
// one 16-byte group a thread suffices, then 32 .. 1024 threads with up to 16 groups (vector)
// or 32 elements (rows whose length is not a multiple of the 16-byte group).
constexpr int kMaxD = 1 << 15;

struct Launch {
    long long blocks, teams;
};
// Teams: as many as the GPU holds at once (per_sm blocks), a multiple of G, at most one per row.
inline Launch plan(long long rows, int G, int tpr, int threads, int per_sm) {
    const long long per = rows / G;
    const int tpb = threads / tpr;
    const long long want = (long long)148 * per_sm * tpb;
    long long S = (want + G - 1) / G;
    if (S > per) S = per;
    if (S < 1) S = 1;
    Launch l;
    l.teams = S * G;
    l.blocks = (l.teams + tpb - 1) / tpb;
    return l;
}

template <int TPR_, int NI_, int VEC_>
struct Cfg {
    static constexpr int TPR = TPR_, NI = NI_, VEC = VEC_;
};
// Calls f(Cfg<..>) with the team for a row of D elements of a type with VEC elements in 16
// bytes.
template <int VEC, typename F>
inline cudaError_t with_team(int D, F&& f) {
    if (D % VEC == 0) {
        const int n = D / VEC;  // 16-byte groups
        if (n <= 8) return f(Cfg<8, 1, VEC>{});
        if (n <= 16) return f(Cfg<16, 1, VEC>{});
        if (n <= 32) return f(Cfg<32, 1, VEC>{});
        if (n <= 64) return f(Cfg<32, 2, VEC>{});
        if (n <= 128) return f(Cfg<64, 2, VEC>{});
        if (n <= 256) return f(Cfg<128, 2, VEC>{});
        if (n <= 512) return f(Cfg<256, 2, VEC>{});
        if (n <= 1024) return f(Cfg<512, 2, VEC>{});
        if (n <= 2048) return f(Cfg<1024, 2, VEC>{});
        if (VEC == 8 || n <= 4096) return f(Cfg<1024, 4, VEC>{});
        if constexpr (VEC == 4) return f(Cfg<1024, 8, VEC>{});
    }
    if (D <= 32) return f(Cfg<32, 1, 1>{});
    if (D <= 128) return f(Cfg<32, 4, 1>{});
    if (D <= 512) return f(Cfg<64, 8, 1>{});
    if (D <= 1024) return f(Cfg<128, 8, 1>{});
    if (D <= 2048) return f(Cfg<256, 8, 1>{});
    if (D <= 4096) return f(Cfg<512, 8, 1>{});
    if (D <= 8192) return f(Cfg<1024, 8, 1>{});
    if (D <= 16384) return f(Cfg<1024, 16, 1>{});
    return f(Cfg<1024, 32, 1>{});
}

template <typename T, typename Tw>
inline cudaError_t launch_fwd(const T* x, const Tw* w, const Tw* b, T* y, float* mean, float* rstd,
                              long long rows, int G, long long inner, int D, float eps,
                              cudaStream_t stream) {
    return with_team<16 / sizeof(T)>(D, [&](auto cfg) {
        using C = decltype(cfg);
        constexpr int threads = block_threads<C::TPR>();
        const Launch l = plan(rows, G, C::TPR, threads, fwd_blocks<C::TPR, C::NI * C::VEC>());
        Shape s{rows, inner, G, D, l.teams, eps};
        ln_fwd_kernel<T, Tw, C::TPR, C::NI, C::VEC>
            <<<(unsigned)l.blocks, threads, 0, stream>>>(x, w, b, y, mean, rstd, s);
        return cudaGetLastError();
    });
}

// Longest row whose sums of dw and db the backward keeps beside it in registers: 8 elements
// a thread at 1024 threads (4 x 8 of the 64 registers a thread has there).
constexpr int kMaxFusedD = 8192;

// Partial sums per group that the backward keeps for a row of D (the S of part).
template <typename T>
inline long long bwd_parts(long long rows, int G, int D) {
    long long S = 0;
    if (D > kMaxFusedD) return rows / G < 64 ? rows / G : 64;
    (void)with_team<16 / sizeof(T)>(D, [&](auto cfg) {
        using C = decltype(cfg);
        constexpr int threads = block_threads<C::TPR>();
        const Launch l = plan(rows, G, C::TPR, threads, bwd_blocks<C::TPR, C::NI * C::VEC>());
        S = G == 1 ? l.blocks : l.teams / G;
        return cudaSuccess;
    });
    return S;
}

template <typename T, typename Tw>
inline cudaError_t launch_bwd(const T* x, const T* dy, const float* mean, const float* rstd,
                              const Tw* w, T* dx, Tw* dw, Tw* db, float* part, long long rows,
                              int G, long long inner, int D, cudaStream_t stream) {
    const bool param = dw || db, fused = D <= kMaxFusedD;
    const long long cols = (long long)G * D, S = bwd_parts<T>(rows, G, D);
    const cudaError_t e = with_team<16 / sizeof(T)>(D, [&](auto cfg) {
        using C = decltype(cfg);
        constexpr int threads = block_threads<C::TPR>();
        const Launch l = plan(rows, G, C::TPR, threads, bwd_blocks<C::TPR, C::NI * C::VEC>());
        Shape s{rows, inner, G, D, l.teams, 0.f};
        const dim3 grid((unsigned)l.blocks);
        if constexpr (C::TPR * C::NI * C::VEC <= kMaxFusedD) {
            if (param) {
                if (C::TPR <= 32 && G == 1)  // (above 32 a block is one team)
                    ln_bwd_kernel<T, Tw, C::TPR, C::NI, C::VEC, true, (C::TPR <= 32)>
                        <<<grid, threads, 0, stream>>>(x, dy, mean, rstd, w, dx, part, s);
                else
                    ln_bwd_kernel<T, Tw, C::TPR, C::NI, C::VEC, true, false>
                        <<<grid, threads, 0, stream>>>(x, dy, mean, rstd, w, dx, part, s);
                return cudaGetLastError();
            }
        }
        ln_bwd_kernel<T, Tw, C::TPR, C::NI, C::VEC, false, false>
            <<<grid, threads, 0, stream>>>(x, dy, mean, rstd, w, dx, part, s);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || !param) return e;
    if (!fused) {
        constexpr int VEC = 16 / sizeof(T);
        const Shape s{rows, inner, G, D, 0, 0.f};
        if (D % VEC == 0)
            ln_bwd_cols_kernel<T, VEC>
                <<<dim3((unsigned)((cols / VEC + 127) / 128), (unsigned)S), 128, 0, stream>>>(
                    x, dy, mean, rstd, part, s);
        else
            ln_bwd_cols_kernel<T, 1><<<dim3((unsigned)((cols + 127) / 128), (unsigned)S), 128, 0,
                                       stream>>>(x, dy, mean, rstd, part, s);
        if (const cudaError_t e2 = cudaGetLastError(); e2 != cudaSuccess) return e2;
    }
    ln_param_kernel<Tw><<<(unsigned)((2 * cols + 31) / 32), 256, 0, stream>>>(part, S, cols, dw, db);
    return cudaGetLastError();
}

}  // namespace ln
}  // namespace wkv7
