// layer_norm.cuh -- layer norm of rows of D elements, forward and backward:
//     mean = sum x / D, rstd = (sum (x - mean)^2 / D + eps)^-1/2, xh = (x - mean) rstd
//     y  = xh w + b
//     dx = rstd (u - sum u / D - xh sum(u xh) / D),  u = dy w
//     dw = sum over rows dy xh,  db = sum over rows dy
// Rows come in G groups with a weight and bias each (one group: layer norm; a group per
// head: the norm of a mixing layer's output): row r is of group (r / inner) % G, inner = 1
// for [.., G, D] rows and T for head-first [B, G, T, D] ones.
//
// Bound by HBM: x once in and y once out (x, dy in, dx out).  A team of threads holds a
// row in registers, so the variance is summed around the mean (no cancellation of two
// large sums) without a second read.  Team t works on rows of group t % G only: w and b stay in
// registers over its rows, and in the backward so do its sums of dw and db, written once at
// the end; a second kernel adds the teams' sums in a fixed order (no atomics: the result
// does not depend on scheduling).  Consecutive teams hold consecutive groups, so a block's
// loads are contiguous for every layout with inner = 1.
//
// All statistics and sums are fp32.  Above 8192 elements the backward's registers no longer
// hold a row and its sums of dw and db, so those get a kernel of their own, which reads x
// and dy again by columns.
#pragma once
#include "common.cuh"

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
    } else if constexpr (VEC == 8) {
        const float4 x = reinterpret_cast<const float4*>(p)[0];
        const float4 y = reinterpret_cast<const float4*>(p)[1];
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
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

// Threads of a block.
template <int TPR> constexpr int block_threads() { return TPR <= 32 ? 128 : TPR; }

// A team of TPR threads holds NI groups of VEC elements a thread.  kTail: D is not a
// multiple of TPR * VEC * NI (groups past D are skipped; VEC divides D).
template <typename T, typename Tw, int TPR, int NI, int VEC>
__global__ void __launch_bounds__(block_threads<TPR>())
ln_fwd_kernel(const T* __restrict__ x, const Tw* __restrict__ w, const Tw* __restrict__ b,
              T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd, Shape s) {
    __shared__ float red[2][1][32];
    const int lane = threadIdx.x % TPR;
    const long long team = (long long)blockIdx.x * (block_threads<TPR>() / TPR) + threadIdx.x / TPR;
    const bool in = team < s.teams;
    const int group = in ? (int)(team % s.G) : 0;
    const long long per = s.rows / s.G, step = s.teams / s.G;
    const float inv = 1.f / (float)s.D;
    // Every team of a block runs as many turns as its first (whole warps stay together
    // for the shuffles); rows past the end are not loaded or stored.
    const long long first = in ? team / s.G : 0;
    const long long turns =
        (per - (long long)blockIdx.x * (block_threads<TPR>() / TPR) / s.G + step - 1) / step;
    float xr[NI][VEC];
    auto fetch = [&](long long k, float (&dst)[NI][VEC]) {
        const bool ok = in && k < per;
        const T* px = x + (ok ? row_at(s, k, group) : 0) * s.D;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (ok && e < s.D) {
                load<VEC>(px + e, dst[i]);
            } else {
#pragma unroll
                for (int q = 0; q < VEC; ++q) dst[i][q] = 0.f;
            }
        }
    };
    long long k = first;
    for (long long turn = 0; turn < turns; ++turn, k += step) {
        fetch(k, xr);
        const bool ok = in && k < per;
        float a[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int q = 0; q < VEC; ++q) a[0] += xr[i][q];
        team_sum<TPR, 1>(a, red[0]);
        const float m = a[0] * inv;
        a[0] = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (e < s.D) {
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    xr[i][q] -= m;
                    a[0] = fmaf(xr[i][q], xr[i][q], a[0]);
                }
            }
        }
        team_sum<TPR, 1>(a, red[1]);
        const float r = 1.f / sqrtf(a[0] * inv + s.eps);
        if (ok) {
            const long long row = row_at(s, k, group);
            T* py = y + row * s.D;
            const long long wo = (long long)group * s.D;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = (i * TPR + lane) * VEC;
                if (e < s.D) {
                    float wv[VEC], bv[VEC];
                    if (w) load<VEC>(w + wo + e, wv);
                    if (b) load<VEC>(b + wo + e, bv);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        float v = xr[i][q] * r;
                        if (w) v *= wv[q];
                        if (b) v += bv[q];
                        xr[i][q] = v;
                    }
                    store<VEC>(py + e, xr[i]);
                }
            }
            if (lane == 0) {
                if (mean) mean[row] = m;
                if (rstd) rstd[row] = r;
            }
        }
    }
}

// part: [S][2][G][D] with S = teams / G, the teams' sums of dy xh and of dy.
template <typename T, typename Tw, int TPR, int NI, int VEC, bool kParam>
__global__ void __launch_bounds__(block_threads<TPR>())
ln_bwd_kernel(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ mean,
              const float* __restrict__ rstd, const Tw* __restrict__ w, T* __restrict__ dx,
              float* __restrict__ part, Shape s) {
    __shared__ float red[2][2][32];
    const int lane = threadIdx.x % TPR;
    const long long team = (long long)blockIdx.x * (block_threads<TPR>() / TPR) + threadIdx.x / TPR;
    const bool in = team < s.teams;
    const int group = in ? (int)(team % s.G) : 0;
    const long long per = s.rows / s.G, step = s.teams / s.G;
    const float inv = 1.f / (float)s.D;
    const long long first = in ? team / s.G : 0;
    const long long turns =
        (per - (long long)blockIdx.x * (block_threads<TPR>() / TPR) / s.G + step - 1) / step;
    const long long wo = (long long)group * s.D;
    float dw[kParam ? NI : 1][VEC], db[kParam ? NI : 1][VEC];
#pragma unroll
    for (int i = 0; i < (kParam ? NI : 1); ++i)
#pragma unroll
        for (int q = 0; q < VEC; ++q) dw[i][q] = db[i][q] = 0.f;
    long long k = first;
    for (long long turn = 0; turn < turns; ++turn, k += step) {
        const bool ok = in && k < per;
        const long long row = ok ? row_at(s, k, group) : 0;
        const float m = ok ? mean[row] : 0.f, r = ok ? rstd[row] : 0.f;
        float xh[NI][VEC], u[NI][VEC];
        float a[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (ok && e < s.D) {
                load<VEC>(x + row * s.D + e, xh[i]);
                load<VEC>(dy + row * s.D + e, u[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (ok && e < s.D) {
                float wv[VEC];
                if (w) load<VEC>(w + wo + e, wv);
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    xh[i][q] = (xh[i][q] - m) * r;
                    if (kParam) {
                        dw[i][q] = fmaf(u[i][q], xh[i][q], dw[i][q]);
                        db[i][q] += u[i][q];
                    }
                    if (w) u[i][q] *= wv[q];
                    a[0] += u[i][q];
                    a[1] = fmaf(u[i][q], xh[i][q], a[1]);
                }
            }
        }
        team_sum<TPR, 2>(a, red[turn & 1]);
        const float c0 = a[0] * inv, c1 = a[1] * inv;
        if (ok) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = (i * TPR + lane) * VEC;
                if (e < s.D) {
#pragma unroll
                    for (int q = 0; q < VEC; ++q) xh[i][q] = r * (u[i][q] - c0 - xh[i][q] * c1);
                    store<VEC>(dx + row * s.D + e, xh[i]);
                }
            }
        }
    }
    if (kParam && in) {
        float* p = part + (team / s.G) * 2 * s.G * s.D + wo;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (e < s.D) {
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    p[e + q] = dw[i][q];
                    p[(long long)s.G * s.D + e + q] = db[i][q];
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
// Teams: as many as fill the GPU a few times over, a multiple of G, at most one per row.
inline Launch plan(long long rows, int G, int tpr, int threads, int per_sm) {
    const long long per = rows / G;
    const int tpb = threads / tpr;
    const long long want = (long long)148 * per_sm * tpb;  // resident teams
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
        const Launch l = plan(rows, G, C::TPR, threads, 2048 / threads);
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
        S = plan(rows, G, C::TPR, threads, 1024 / threads).teams / G;
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
        const Launch l = plan(rows, G, C::TPR, threads, 1024 / threads);
        Shape s{rows, inner, G, D, l.teams, 0.f};
        if constexpr (C::TPR * C::NI * C::VEC <= kMaxFusedD) {
            if (param) {
                ln_bwd_kernel<T, Tw, C::TPR, C::NI, C::VEC, true>
                    <<<(unsigned)l.blocks, threads, 0, stream>>>(x, dy, mean, rstd, w, dx, part, s);
                return cudaGetLastError();
            }
        }
        ln_bwd_kernel<T, Tw, C::TPR, C::NI, C::VEC, false>
            <<<(unsigned)l.blocks, threads, 0, stream>>>(x, dy, mean, rstd, w, dx, part, s);
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
