// la_recurrent.cuh -- one pass of the decay linear attention token by token on CUDA cores,
// fp32 throughout: the path of fp32 inputs and of head size 256, and the anchor that the
// tensor-core kernel is checked against.
//
//     U <- d_t U + y_t z_t^T;   out_t = U^T x_t        (la_common.cuh)
//
// Unlike the delta rule, a token's update does not read the state, so tokens only meet in
// an elementwise multiply-add: nothing but the issue rate of the 3 D^2 fp32 operations per
// token bounds a block, and shared memory must feed them.  A block owns 64 columns of one
// (segment, head); a thread holds a tile of 16 rows x 4 columns (64 registers), so the 8
// float4 of x and y that it reads per token serve 192 operations (one column per thread
// would read as many for 48).  The D / 16 row parts of a column are adjacent lanes; their
// sums meet by shuffles.  Parts of a staged row are 20 floats apart, so the parts that
// read together sit in different banks.
//
// fp32, B = 2, T = 333, H = 8 of 64: 115 us in one chain per head (0.34 us a token), 32 us in
// 32-token segments.  B = 8, T = 4096, H = 64 here: bf16 4.75 ms (3.53 ms, and 1.22 ms for its
// segments' states: the plan cuts it, which does not pay there), fp32 2.96 ms (2.12 + 0.82);
// 0.72 ms is the issue rate's floor.  Head size 256, 8 x 4096 tokens of 16 heads, bf16: 12.5 ms.
//
// Tokens are staged in tiles (fp32, the decay's exponential taken once); the next tile's
// global loads are in registers while the current one runs.  Outputs leave through
// shared memory so that rows are written whole, and their dot products with another
// tensor (the decay's gradient) cost one warp reduction per token and not one per thread.
#pragma once
#include "la_common.cuh"

namespace wkv7 {
namespace la {

template <int D>
struct RecCfg {
    static constexpr int kThreads = D;
    static constexpr int kParts = D / 16;      // row parts of a column
    static constexpr int kSlabs = D / 64;      // 64-column slabs
    static constexpr int kRow = kParts * 20;   // floats of a staged row
    static constexpr int kTile = D == 256 ? 8 : 16;
};

// State entry (row, col .. col + 3) as float4 from [row][col] or, transposed, [col][row].
template <int D>
__device__ __forceinline__ void load_tile(const float* s, bool transposed, int row0, int col0,
                                          float4 (&S)[16]) {
    if (!transposed) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            S[i] = *reinterpret_cast<const float4*>(s + (row0 + i) * D + col0);
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            float4 c[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                c[q] = *reinterpret_cast<const float4*>(s + (col0 + q) * D + row0 + i);
            S[i + 0] = make_float4(c[0].x, c[1].x, c[2].x, c[3].x);
            S[i + 1] = make_float4(c[0].y, c[1].y, c[2].y, c[3].y);
            S[i + 2] = make_float4(c[0].z, c[1].z, c[2].z, c[3].z);
            S[i + 3] = make_float4(c[0].w, c[1].w, c[2].w, c[3].w);
        }
    }
}
template <int D>
__device__ __forceinline__ void store_tile(float* s, int row0, int col0, const float4 (&S)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) *reinterpret_cast<float4*>(s + (row0 + i) * D + col0) = S[i];
}

template <typename Tin, int D, bool kRev, bool kStateOnly>
__global__ void __launch_bounds__(D)
la_recurrent_kernel(const Pass<Tin> p) {
    using C = RecCfg<D>;
    constexpr int kThreads = C::kThreads, kTile = C::kTile;
    constexpr int kXY = kTile * D / 4 / kThreads;    // groups of 4 of x (and y) per thread
    constexpr int kZ = kTile * 16 / kThreads;        // and of z (0 or more)
    constexpr int kZmax = kZ > 0 ? kZ : 1;
    __shared__ __align__(16) float sx[kStateOnly ? 1 : kTile][C::kRow];
    __shared__ __align__(16) float sy[kTile][C::kRow];
    __shared__ __align__(16) float sz[kTile][64];
    __shared__ __align__(16) float so[kStateOnly ? 1 : kTile][64];
    __shared__ float sd[kTile];
    __shared__ uint8_t slive[kTile];
    __shared__ float red[kThreads / 32];
    const Geom& G = p.geom;
    const int tid = threadIdx.x;
    if (!seqlens_ok(G, tid, kThreads)) {
        if (tid == 0 && blockIdx.x == 0) raise_flag(5 /* WKV7_ERR_DEVICE_BAD_SEQLENS */);
        return;
    }
    const int slab = (int)(blockIdx.x % C::kSlabs);
    const long long sh = blockIdx.x / C::kSlabs;
    const int h = (int)(sh % G.H);
    const long long slot = sh / G.H;
    const Item it = locate(G, (int)slot, p.seg);
    if (it.n < 0) return;
    // a state-only pass runs the segments whose state a later one (in the pass's
    // direction) starts from
    if (kStateOnly && (kRev ? it.j == 0 : it.j == it.nseg - 1)) return;
    const int tb = it.j * p.seg, te = min(it.len, tb + p.seg);  // tokens [tb, te)
    const Rows rw = rows_of(G, it, h);
    const uint8_t* mrow = p.mask ? p.mask + (long long)it.bb * G.T + it.bos : nullptr;
    const float ghead = p.g_per_head ? to_f32(p.g[h]) : 0.f;

    const int part = tid % C::kParts, cg = tid / C::kParts;
    const int row0 = 16 * part, col0 = 64 * slab + 4 * cg;
    const long long state_at = ((long long)it.n * G.H + h) * D * D;
    float4 S[16];
    if (!kStateOnly && p.init) {
        const float* s = p.init + (p.init_by_slot ? (slot * G.H + h) * D * D : state_at);
        load_tile<D>(s, p.init_transposed, row0, col0, S);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    // Tile k of the pass covers cnt tokens from t0 (forward) or up to t0 (backward);
    // local token i of it is t0 + i or t0 - i.  Tiles never cross a chunk.
    //
    // A decay's rounding to fp32 is the same at every token of a constant decay, so a state
    // 4096 tokens old would be off by 4096 half steps.  The first decay of every tile
    // therefore takes what the tile's others and the earlier ones are off by (their
    // product against the exponential in 64 bits), and the product over any stretch
    // stays within a tile's roundings of the exact one.
    float4 rx[kXY], ry[kXY], rz[kZmax];
    float rd = 1.f;
    bool rl = true;
    double off = 1.0, logtot = 0.0;
    const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
    auto token = [&](int t0, int i) { return kRev ? t0 - i : t0 + i; };
    auto fetch = [&](int t0, int cnt) {
#pragma unroll
        for (int u = 0; u < kXY; ++u) {
            const int idx = tid + u * kThreads, i = idx / (D / 4), e = 4 * (idx % (D / 4));
            ry[u] = zero4;
            if (!kStateOnly) rx[u] = zero4;
            if (i < cnt) {
                const int t = token(t0, i);
                const long long at = (rw.first + t * rw.step) * D + e;
                if (kRev || !mrow || mrow[t]) ry[u] = load4(p.y + at);
                if (!kStateOnly) rx[u] = load4(p.x + at);
            }
        }
#pragma unroll
        for (int u = 0; u < kZmax; ++u) {
            const int idx = tid + u * kThreads, i = idx / 16, e = 4 * (idx % 16);
            rz[u] = zero4;
            if (i < cnt) {
                const int t = token(t0, i);
                const long long at = (rw.first + t * rw.step) * D + 64 * slab + e;
                if (kRev || !mrow || mrow[t]) rz[u] = load4(p.z + at);
            }
        }
        if (tid < 32) {  // the tile's decays, one token a lane (kTile <= 16)
            float gd = 0.f;
            rl = false;
            if (tid < cnt) {
                const int t = token(t0, tid);
                rl = !mrow || mrow[t];
                if (rl)
                    gd = clamp_log_decay(p.g_per_head ? ghead : to_f32(p.g[rw.first + t * rw.step]));
            }
            rd = expf(gd);
            const bool plain = rd > 1e-30f && rd < 1e30f;
            const double e = plain ? exp((double)gd) / (double)rd : 1.0;
            double others = tid == 0 ? 1.0 : e;
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) others *= __shfl_xor_sync(0xffffffffu, others, m);
            if (tid == 0) {
                const double want = off * others * e * (double)rd;
                rd = (float)want;
                off = plain && rd > 1e-30f ? want / (double)rd : 1.0;
            }
            if (kStateOnly) {
                double sum = gd;
#pragma unroll
                for (int m = 8; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                logtot += sum;
            }
        }
    };
    auto put = [&](int cnt) {
#pragma unroll
        for (int u = 0; u < kXY; ++u) {
            const int idx = tid + u * kThreads, i = idx / (D / 4), e = 4 * (idx % (D / 4));
            const int at = (e / 16) * 20 + e % 16;
            float4 y = ry[u];
            if (kRev) {
                y.x *= p.key_scale;
                y.y *= p.key_scale;
                y.z *= p.key_scale;
                y.w *= p.key_scale;
            }
            *reinterpret_cast<float4*>(&sy[i][at]) = y;
            if (!kStateOnly) *reinterpret_cast<float4*>(&sx[i][at]) = rx[u];
        }
#pragma unroll
        for (int u = 0; u < kZmax; ++u) {
            const int idx = tid + u * kThreads, i = idx / 16, e = 4 * (idx % 16);
            if (i < kTile) *reinterpret_cast<float4*>(&sz[i][e]) = rz[u];
        }
        if (tid < cnt) {
            sd[tid] = rd;
            slive[tid] = rl;
        }
    };
    // first token of the next tile after one of cnt tokens from t0, and its length
    auto tile_len = [&](int t0) {
        if (kRev) {
            const int lo = max(tb, t0 & ~(kTile - 1));  // tiles end at multiples of kTile
            return t0 - lo + 1;
        }
        return min(kTile, te - t0);
    };

    float dprev = 1.f;   // backward: the decay between the token before and this one
    int t0 = kRev ? te - 1 : tb;
    int cnt = te > tb ? tile_len(t0) : 0;
    if (cnt > 0) fetch(t0, cnt);
    while (cnt > 0) {
        __syncthreads();  // the last tile's readers are done
        put(cnt);
        __syncthreads();
        const int cur = t0, n_cur = cnt;
        t0 = kRev ? t0 - cnt : t0 + cnt;
        cnt = (kRev ? t0 >= tb : t0 < te) ? tile_len(t0) : 0;
        if (cnt > 0) fetch(t0, cnt);

        // backward: <S_end, G_end> when the tile opens a chunk
        if (kRev && !kStateOnly && p.ck_dot &&
            (cur == it.len - 1 || (cur & (kRecChunk - 1)) == kRecChunk - 1)) {
            const long long at =
                (slot_of(G, it, cur / kRecChunk, kRecChunk) * G.H + h) * C::kSlabs + slab;
            const float4* ck = static_cast<const float4*>(p.ck) + at * 16 * kThreads + tid;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 c = ck[i * kThreads];
                s += c.x * S[i].x + c.y * S[i].y + c.z * S[i].z + c.w * S[i].w;
            }
            s *= dprev;
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
            if ((tid & 31) == 0) red[tid >> 5] = s;
            __syncthreads();
            if (tid == 0) {
                s = 0.f;
#pragma unroll
                for (int i = 0; i < kThreads / 32; ++i) s += red[i];
                p.ck_dot[at] = s;
            }
        }

        for (int i = 0; i < n_cur; ++i) {
            const float d = kRev ? dprev : sd[i];
            if (kRev) dprev = sd[i];
            const float4 z = *reinterpret_cast<const float4*>(&sz[i][4 * cg]);
            float4 acc = zero4;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 y4 = *reinterpret_cast<const float4*>(&sy[i][20 * part + 4 * q]);
                const float yv[4] = {y4.x, y4.y, y4.z, y4.w};
                float4 x4 = zero4;
                if (!kStateOnly) x4 = *reinterpret_cast<const float4*>(&sx[i][20 * part + 4 * q]);
                const float xv[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float4& s = S[4 * q + r];
                    s.x = fmaf(d, s.x, yv[r] * z.x);
                    s.y = fmaf(d, s.y, yv[r] * z.y);
                    s.z = fmaf(d, s.z, yv[r] * z.z);
                    s.w = fmaf(d, s.w, yv[r] * z.w);
                    if (!kStateOnly) {
                        acc.x = fmaf(s.x, xv[r], acc.x);
                        acc.y = fmaf(s.y, xv[r], acc.y);
                        acc.z = fmaf(s.z, xv[r], acc.z);
                        acc.w = fmaf(s.w, xv[r], acc.w);
                    }
                }
            }
            if (!kStateOnly) {
#pragma unroll
                for (int m = 1; m < C::kParts; m <<= 1) {
                    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, m);
                    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, m);
                    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, m);
                    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, m);
                }
                if (part == 0) *reinterpret_cast<float4*>(&so[i][4 * cg]) = acc;
            }
        }

        if (!kStateOnly) {
            __syncthreads();
            for (int i = tid >> 5; i < n_cur; i += kThreads / 32) {
                const int lane = tid & 31;
                const long long row = rw.first + token(cur, i) * rw.step;
                const long long at = row * D + 64 * slab + 2 * lane;
                float2 o = *reinterpret_cast<const float2*>(&so[i][2 * lane]);
                o.x *= p.inter_scale;
                o.y *= p.inter_scale;
                const bool none = kRev && !slive[i];
                if (none) o = make_float2(0.f, 0.f);
                if (p.dots) {
                    float s = 0.f;
                    if (!none) {
                        const float2 w = load2(p.dot_with + at);
                        s = o.x * w.x + o.y * w.y;
                    }
#pragma unroll
                    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                    if (lane == 0)
                        p.dots[slab * p.dots_stride + scratch_of(G, it, h, token(cur, i))] = s;
                }
                p.out[at] = from_f32<Tin>(o.x);
                p.out[at + 1] = from_f32<Tin>(o.y);
            }
            // forward: keep the state at the end of a chunk
            const int last = cur + n_cur - 1;
            if (!kRev && p.ck && (last == it.len - 1 || (last & (kRecChunk - 1)) == kRecChunk - 1)) {
                const long long at =
                    (slot_of(G, it, last / kRecChunk, kRecChunk) * G.H + h) * C::kSlabs + slab;
                float4* ck = static_cast<float4*>(p.ck) + at * 16 * kThreads + tid;
#pragma unroll
                for (int i = 0; i < 16; ++i) ck[i * kThreads] = S[i];
            }
        }
    }
    if (kRev) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            S[i].x *= dprev;
            S[i].y *= dprev;
            S[i].z *= dprev;
            S[i].w *= dprev;
        }
    }
    if (kStateOnly) {
        store_tile<D>(p.seg_state + (slot * G.H + h) * D * D, row0, col0, S);
        if (tid == 0 && slab == 0) p.seg_decay[slot * G.H + h] = (float)exp(logtot);
    } else if (p.fin && (kRev ? it.j == 0 : it.j == it.nseg - 1)) {
        store_tile<D>(p.fin + state_at, row0, col0, S);
    }
}

template <typename Tin, int D, bool kRev, bool kStateOnly>
inline cudaError_t launch_recurrent_d(const Pass<Tin>& p, cudaStream_t stream) {
    const long long blocks = p.geom.slots(p.seg) * p.geom.H * RecCfg<D>::kSlabs;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    la_recurrent_kernel<Tin, D, kRev, kStateOnly><<<(unsigned)blocks, D, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename Tin, bool kRev, bool kStateOnly>
inline cudaError_t launch_recurrent_pass(const Pass<Tin>& p, int D, cudaStream_t stream) {
    return D == 64    ? launch_recurrent_d<Tin, 64, kRev, kStateOnly>(p, stream)
           : D == 128 ? launch_recurrent_d<Tin, 128, kRev, kStateOnly>(p, stream)
                      : launch_recurrent_d<Tin, 256, kRev, kStateOnly>(p, stream);
}

}  // namespace la
}  // namespace wkv7
