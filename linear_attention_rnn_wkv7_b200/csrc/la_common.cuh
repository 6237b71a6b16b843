// la_common.cuh -- linear attention with one decay per head (no delta rule): the pieces
// that its kernels share.
//
// Per (sequence, head), with a D x D state S stored [k][v] and a log decay g_t:
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,      o_t = scale S_t^T q_t.
// A token whose mask is 0 leaves the state as it is and reads it.
//
// One operator serves the forward and the whole backward.  Call out = A(x, y, z) the map
//     U_t = e^{g_t} U_{t-1} + y_t z_t^T,      out_t = U_t^T x_t,
// and A' the same run backwards in time (U_t = y_t z_t^T + e^{g_{t+1}} U_{t+1}).  Then, up
// to the scale,
//     o = A(q, k, v)       from S_0                          (state S)
//     dq = A(do, v, k)     from S_0^T                        (state S^T)
//     dv = A'(k, q, do)    from dS_T                         (state G = dL/dS)
//     dk = A'(v, do, q)    from dS_T^T                       (state G^T)
// so a pass is described by its three inputs, its direction and the layout of its
// initial state.  The gradient of the log decays follows from the pairs (t, s):
// with c_t the prefix sum of g inside a chunk, o_t holds e^{c_t - c_s}, hence
//     dL/dc_t = q_t . dq_t - k_t . dk_t,
//     dg_t = sum of dL/dc_s over the chunk's s >= t, + <S_end, G_end> of the chunk,
// where G_end is the gradient that reaches the chunk's last state from later tokens.
// Restarting the sum at every chunk keeps it as exact as one chunk's terms (the sum's errors
// grow with its length, and where memories are short dg does not).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace wkv7 {
namespace la {

// Tokens per chunk of the tensor-core kernel; its segments are multiples of it, the recurrent
// kernel's of kRecChunk.
constexpr int kChunk = 128;
// Spacing of the states that the recurrent kernel keeps for dg: fp32 results want shorter
// sums than bf16's (summed over the tokens of 900, with memories of 3 to 30 tokens, dg was
// 1.2e-5 off at 128 and is a quarter of that at 32).
constexpr int kRecChunk = 32;

// Log decays below this are taken as it: e^-120 is 0 in fp32 next to any state, and prefix
// sums stay finite (g = -inf resets the state).  NaN stays NaN.
__device__ __forceinline__ float clamp_log_decay(float g) { return g < -120.f ? -120.f : g; }

// Where a sequence's tokens are, and how it is cut into segments of `seg` tokens.  Slot
// floor(start / seg) + n + j holds segment j of sequence n (the slots of different
// sequences never overlap); unpacked problems have exactly nseg slots a sequence.
struct Geom {
    const int32_t* cu;  // packed sequences' offsets, or nullptr
    int T, N, H;
    int head_first;

    __host__ __device__ long long slots(int seg) const {
        if (cu) return (long long)T / seg + N;
        return (long long)N * segs(T, seg);
    }
    __host__ __device__ static int segs(int len, int seg) {
        return len <= seg ? 1 : (len - 1) / seg + 1;
    }
};

struct Item {
    int n, j;       // sequence, segment (n < 0: the slot is empty)
    int nseg;       // segments of the sequence
    int bos, len;   // first token row (packed) and length of the sequence
    int bb;         // batch row of the inputs
};

// Whether sequence i's offsets are out of order or range, or the first is not 0.
__host__ __device__ __forceinline__ bool seqlen_bad(const Geom& g, int i) {
    const int a = g.cu[i], b = g.cu[i + 1];
    return (a < 0) | (b < a) | (b > g.T) | ((i == 0) & (a != 0));
}
// Whether cu_seqlens is non-decreasing from 0 within [0, T]; every thread of the block calls it.
__device__ __forceinline__ bool seqlens_ok(const Geom& g, int tid, int threads) {
    if (!g.cu) return true;
    int bad = 0;
    for (int i = tid; i < g.N; i += threads) bad |= seqlen_bad(g, i);
    return !__syncthreads_or(bad);
}

// (Slot numbers fit 32 bits: the entry points check.)
__host__ __device__ __forceinline__ Item locate(const Geom& g, int slot, int seg) {
    Item it;
    if (!g.cu) {
        it.nseg = Geom::segs(g.T, seg);
        it.n = slot / it.nseg;
        it.j = slot - it.n * it.nseg;
        it.bos = 0;
        it.len = g.T;
        it.bb = it.n;
        return it;
    }
    int lo = 0, hi = g.N;  // the last n with floor(cu[n] / seg) + n <= slot
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.cu[mid] / seg + mid <= slot) lo = mid; else hi = mid;
    }
    it.n = lo;
    it.bos = g.cu[lo];
    it.len = g.cu[lo + 1] - it.bos;
    it.j = slot - it.bos / seg - lo;
    it.nseg = Geom::segs(it.len, seg);
    it.bb = 0;
    // between two sequences' slots, or (offsets that do not begin at 0) before the first's
    if (it.j < 0 || it.j >= it.nseg) it.n = -1;
    return it;
}
__device__ __forceinline__ long long slot_of(const Geom& g, const Item& it, int j, int seg) {
    if (!g.cu) return (long long)it.n * Geom::segs(g.T, seg) + j;
    return (long long)it.bos / seg + it.n + j;
}

// Row of token t of head h: first + t * step, in [.., D] tensors and in [.., 1] scalars.
struct Rows {
    long long first, step;
};
__device__ __forceinline__ Rows rows_of(const Geom& g, const Item& it, int h) {
    Rows r;
    if (g.head_first) {
        r.first = ((long long)it.bb * g.H + h) * g.T + it.bos;
        r.step = 1;
    } else {
        r.first = ((long long)it.bb * g.T + it.bos) * g.H + h;
        r.step = g.H;
    }
    return r;
}

// Index of token t of head h in scratch values of one per token and head: head first whatever
// the layout, so that a chunk's are contiguous.
__device__ __forceinline__ long long scratch_of(const Geom& g, const Item& it, int h, int t) {
    return ((long long)it.bb * g.H + h) * g.T + it.bos + t;
}

// One pass: out = A(x, y, z) or A'(x, y, z).
template <typename Tin>
struct Pass {
    Geom geom;
    const Tin *x, *y, *z;
    const Tin* g;         // [.., H] for each token, or [H]
    int g_per_head;
    const uint8_t* mask;  // [B, T] or nullptr
    // forward direction: masked tokens write nothing (y, z are not used there);
    // backward direction: they get no output (it is written as 0)
    Tin* out;
    float pair_scale;     // on y_t z_t^T inside out (the score part)
    float inter_scale;    // on what the state before the chunk gives to out
    float key_scale;      // on y_t z_t^T inside the state
    int parts;            // bf16 parts of the state update's operand (tensor cores): 3 where the
                          // state itself is a result, 2 where it only makes bf16 results
    int run;              // > 0: chunks per block, see Schedule (tensor-core kernel); else segments
    float* ho_state;      // [block][D * D], and
    unsigned* ho_flag;    // [block][8], zero: states handed from block to block
    int seg;              // tokens per segment
    const float* init;    // states before the first token: [N][H][D][D], or by slot when
    int init_by_slot;     // init_by_slot; nullptr: zeros
    int init_transposed;  // init holds [z][y] instead of [y][z]
    float* fin;           // final states [N][H][D][D] as [y][z], or nullptr
    // state-only passes: each segment's own state and e^{sum of g}
    float* seg_state;     // [slot][H][D][D]
    float* seg_decay;     // [slot][H]
    // gradient of the log decays
    const Tin* dot_with;  // dots = dot_with[row] . out[row] before rounding, one for each
    float* dots;          // [slab][B][H][T]
    long long dots_stride;
    void* ck;             // states at each chunk's end (layout private to the kernel)
    float* ck_dot;        // [chunk slot][H][parts]: parts of <ck, state before the chunk>
    unsigned wait_ns;     // limit of a wait of the tensor-core kernel, and (test hook) whether one
    int handoff_at_once;  // for a state handed on gives up at its first look
};

// ---- start states of the segments --------------------------------------------------------
// seg_state[slot] holds the state that segment j makes from zero; it becomes the state
// before segment j.  One thread per state entry walks over the segments in the direction
// of the pass: S <- decay_j S + local_j.  (init [N][H][D*D] or nullptr.)
template <bool kRev>
__global__ void __launch_bounds__(256)
la_chain_kernel(Geom g, const float* __restrict__ init, float* __restrict__ seg_state,
                const float* __restrict__ seg_decay, int seg, int DD) {
    if (!seqlens_ok(g, threadIdx.x, 256)) return;
    const long long per = DD / 4;  // float4 per state
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)g.N * g.H * per) return;
    const long long unit = i / per;
    const int e = (int)(i - unit * per);
    const int n = (int)(unit / g.H), h = (int)(unit - (long long)n * g.H);
    Item it;
    it.n = n;
    it.bos = g.cu ? g.cu[n] : 0;
    it.len = g.cu ? g.cu[n + 1] - it.bos : g.T;
    const int nseg = Geom::segs(it.len, seg);
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (init) S = reinterpret_cast<const float4*>(init)[i];
    const long long base = slot_of(g, it, 0, seg);
    // four segments' own states in flight at a time
    for (int j0 = 0; j0 < nseg; j0 += 4) {
        float4 loc[4];
        float d[4];
        float4* at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int jj = j0 + u, j = kRev ? nseg - 1 - jj : jj;
            const long long slot = (base + j) * g.H + h;
            at[u] = reinterpret_cast<float4*>(seg_state) + slot * per + e;
            if (jj < nseg - 1) {  // (nothing starts from the last one's)
                loc[u] = *at[u];
                d[u] = seg_decay[slot];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (j0 + u >= nseg) break;
            *at[u] = S;
            if (j0 + u == nseg - 1) break;
            S.x = fmaf(d[u], S.x, loc[u].x);
            S.y = fmaf(d[u], S.y, loc[u].y);
            S.z = fmaf(d[u], S.z, loc[u].z);
            S.w = fmaf(d[u], S.w, loc[u].w);
        }
    }
}

// ---- gradient of the log decays ------------------------------------------------------------
// One warp per (chunk of kC tokens, head), kC / 32 tokens a lane: dL/dc = (q . dq) - (k . dk), summed from
// the chunk's end, plus the chunk's <S_end, G_end>.  dg [.., H] per token, or part
// [chunk slot][H], the chunk's sum, for decays shared by all tokens of a head.
template <typename Tin, int kC>
__global__ void __launch_bounds__(128)
la_dg_kernel(Geom g, const uint8_t* __restrict__ mask, const float* __restrict__ qdq,
             const float* __restrict__ kdk, int slabs, long long stride,
             const float* __restrict__ ends, int nends, Tin* __restrict__ dg,
             float* __restrict__ part) {
    if (!seqlens_ok(g, threadIdx.x, 128)) return;
    constexpr int kPer = kC / 32;
    const int lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const long long slots = g.slots(kC);
    if (id >= slots * g.H) return;
    const long long slot = id / g.H;
    const int h = (int)(id - slot * g.H);
    const Item it = locate(g, (int)slot, kC);
    if (it.n < 0) {
        if (part && lane == 0) part[id] = 0.f;
        return;
    }
    const Rows rw = rows_of(g, it, h);
    const int t0 = it.j * kC + kPer * lane;
    float v[kPer];
    bool live[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int t = t0 + i;
        v[i] = 0.f;
        live[i] = t < it.len;
        if (live[i]) {
            const long long at = scratch_of(g, it, h, t);
            for (int s = 0; s < slabs; ++s) v[i] += qdq[s * stride + at] - kdk[s * stride + at];
            if (mask) live[i] = mask[(long long)it.bb * g.T + it.bos + t] != 0;
        }
    }
#pragma unroll
    for (int i = kPer - 2; i >= 0; --i) v[i] += v[i + 1];
    float after = 0.f, run = v[0];  // sum of the lanes after this one
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float o = __shfl_down_sync(0xffffffffu, run, m);
        if (lane + m < 32) run += o;
    }
    after = __shfl_down_sync(0xffffffffu, run, 1);
    if (lane == 31) after = 0.f;
    for (int s = 0; s < nends; ++s) after += ends[id * nends + s];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const float x = live[i] ? v[i] + after : 0.f;
        sum += x;
        if (dg && t0 + i < it.len) dg[rw.first + (t0 + i) * rw.step] = from_f32<Tin>(x);
    }
    if (part) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (lane == 0) part[id] = sum;
    }
}

// dg[h] = sum of part[slot][h] over the slots, in a fixed order: one block per head.
template <typename Tin>
__global__ void __launch_bounds__(256)
la_dg_sum_kernel(Geom g, const float* __restrict__ part, long long slots, Tin* __restrict__ dg) {
    __shared__ float red[8];
    if (!seqlens_ok(g, threadIdx.x, 256)) return;
    const int h = blockIdx.x;
    float s = 0.f;
    for (long long i = threadIdx.x; i < slots; i += 256) s += part[i * g.H + h];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += red[i];
        dg[h] = from_f32<Tin>(s);
    }
}

// ---- rows behind the last sequence ---------------------------------------------------------
// Zeros in the rows behind the last packed sequence of up to three [.., D] tensors and one of a
// value per token and head; nullptr: none.  They are one stretch of memory (token-major) or one
// a head; D-wide rows are whole 16-byte groups.
template <typename Tin>
struct Tail {
    Tin* x[3];
    Tin* s;
    int D;
};
template <typename Tin>
__global__ void __launch_bounds__(256) la_tail_kernel(Geom g, Tail<Tin> t) {
    if (!seqlens_ok(g, threadIdx.x, 256)) return;
    constexpr int kVec = 16 / sizeof(Tin);
    const long long end = g.N > 0 ? g.cu[g.N] : 0;
    const int parts = g.head_first ? g.H : 1;
    const long long width = g.head_first ? 1 : g.H;          // values of a token in a part
    const long long n = (g.T - end) * width, at = end * width, stride = g.T * width;
    const long long first = (long long)blockIdx.x * 256 + threadIdx.x, step = (long long)gridDim.x * 256;
    for (int i = 0; i < 3; ++i) {
        if (!t.x[i]) continue;
        const long long v = n * (t.D / kVec);
        for (int h = 0; h < parts; ++h) {
            uint4* to = reinterpret_cast<uint4*>(t.x[i] + (h * stride + at) * t.D);
            for (long long e = first; e < v; e += step) to[e] = make_uint4(0, 0, 0, 0);
        }
    }
    if (t.s)
        for (int h = 0; h < parts; ++h)
            for (long long e = first; e < n; e += step) t.s[h * stride + at + e] = from_f32<Tin>(0.f);
}

}  // namespace la
}  // namespace wkv7
