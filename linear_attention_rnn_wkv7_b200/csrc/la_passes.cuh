// la_passes.cuh -- host side of the decay linear attention: how a problem is cut into
// segments, the workspace, and the passes of the forward and the backward (la_common.cuh).
#pragma once
#include <algorithm>

#include "la_common.cuh"
#include "la_chunked.cuh"
#include "la_recurrent.cuh"

namespace wkv7 {
namespace la {

struct Problem {
    Geom geom;
    int B, D;
    bool bf16, chunked;
    unsigned wait_ns = 1000000000u;  // a second; less, and the next, by a test hook alone
    int handoff_at_once = 0;
    long long rows() const { return (long long)B * geom.T * geom.H; }
    // spacing of the states kept for dg
    int ck_every() const { return chunked ? kChunk : kRecChunk; }
    // column slabs that one (segment, head) is split into
    int slabs() const { return chunked ? 1 : D / 64; }
    // parts of a chunk's <S_end, G_end>
    int ends() const { return chunked ? D / 16 : D / 64; }
};

// How the work is laid out on the GPU.  One segment per sequence needs nothing extra.  With fewer
// (sequence, head) units than the GPU holds blocks, sequences are cut: a pass over y and z first
// gives every segment's own state (half of a pass's reads, no outputs), la_chain_kernel
// joins them, and all segments run at once.  The estimate counts time on the longest block in
// grains, 128 tokens for the tensor-core kernel (2 to 4 us) and 32 for the recurrent one (about
// 10 us): a segment costs its grains and its state's way in and out, a state-only pass 0.6 of a
// full one, the join and the launches the rest (16384 tokens x 16 heads of 128: 64 segments
// 414 us, the 9 that this picks 144 us; fp32 333 tokens x 16 units: uncut 115 us).  With more
// units than blocks the tensor-core kernel takes runs (la_chunked.cuh, Schedule) instead.
struct Plan {
    int seg;
    bool split;
    int run;           // > 0: chunks per block
    long long blocks;  // of the runs
};
// SMs of a B200: a plan, and with it the workspace's size, is the same on every device, and a
// query needs none.  (With fewer SMs runs only take turns: blocks start in order.)
constexpr int kBlocks = 148;

inline Plan make_plan(const Problem& p) {
    const Geom& g = p.geom;
    // blocks that run at once: one per SM (tensor cores) or by registers (64 a state tile)
    const long long resident = p.chunked ? kBlocks : (long long)kBlocks * 384 / p.D;
    // segments are whole grains; costs in grains of time
    const int grain = p.chunked ? kChunk : kRecChunk;
    const double per_segment = p.chunked ? 2.0 : 0.3, launches = p.chunked ? 4.0 : 0.6,
                 join = p.chunked ? 0.35 : 0.05;
    const long long chunks = std::max<long long>(1, ((long long)g.T + grain - 1) / grain);
    Plan best{(int)(chunks * grain), false, 0, 0};
    if (chunks * grain > 0x7fffff80LL) best.seg = 0x7fffff80;
    const long long units = (long long)g.N * g.H * p.slabs();
    const long long all = g.slots(kChunk) * g.H;
    // Whole sequences round robin keep neighbouring heads, whose rows share DRAM pages, at work
    // together: 512 sequences of one length, 3.46 rounds' work in 4 rounds, take 327 us so and
    // 347 us in runs.  Runs are for what fills its rounds worse, and for packed lengths.  (A
    // packed sequence longer than a run is worked on by its blocks in turn: 60000 of 69565 tokens
    // in one of 64 sequences, 32 heads, 970 us, where even lengths take 409 us.)
    const long long rounds = (units + kBlocks - 1) / kBlocks;
    if (p.chunked && !g.cu && units * 5 >= rounds * kBlocks * 4) return best;
    if (p.chunked && units > kBlocks && all <= 0x7fffffffLL) {
        const long long even = (all + kBlocks - 1) / kBlocks;
        best.run = (int)(g.cu ? even : std::max(chunks, even));
        best.blocks = (all + best.run - 1) / best.run;
        return best;
    }
    if (chunks < 4 || units == 0) return best;
    if (g.cu) {
        // lengths are on the device: cut only sequences longer than an even share
        const long long share = chunks * g.H * p.slabs() / resident;
        const long long c = std::max<long long>(4, share);
        if (c < chunks) best = Plan{(int)(c * grain), true, 0, 0};
        return best;
    }
    double least = (double)((units + resident - 1) / resident) * ((double)chunks + per_segment);
    for (long long n = 2; n <= std::min<long long>(chunks, 256); ++n) {
        const long long c = (chunks + n - 1) / n, used = (chunks + c - 1) / c;
        const double waves = (double)((units * used + resident - 1) / resident);
        const double t = waves * (1.6 * (double)c + 2 * per_segment) + join * (double)used + launches;
        if (used > 1 && t < least) {
            least = t;
            best = Plan{(int)(c * grain), true, 0, 0};
        }
    }
    return best;
}

// Workspace pieces, in floats, each rounded up to 256 bytes.
struct Carve {
    size_t at = 0;
    size_t take(size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~(size_t)255;
        return here;
    }
};
struct Segs {
    size_t state = 0, decay = 0;
};
inline Segs carve_segs(Carve& c, const Problem& p, const Plan& plan) {
    Segs s;
    if (!plan.split) return s;
    const size_t n = (size_t)p.geom.slots(plan.seg) * p.geom.H;
    s.state = c.take(n * p.D * p.D * sizeof(float));
    s.decay = c.take(n * sizeof(float));
    return s;
}
// States handed from block to block, and their flags for `passes` passes.
struct Handoff {
    size_t state = 0, flags = 0, flag_bytes = 0;
};
inline Handoff carve_handoff(Carve& c, const Problem& p, const Plan& plan, int passes) {
    Handoff h;
    if (plan.run == 0) return h;
    h.state = c.take((size_t)plan.blocks * p.D * p.D * sizeof(float));
    h.flag_bytes = (size_t)passes * plan.blocks * 8 * sizeof(unsigned);
    h.flags = c.take(h.flag_bytes);
    return h;
}
template <typename Tin>
inline void use_handoff(Pass<Tin>& a, const Plan& plan, const Handoff& h, uint8_t* ws, int pass) {
    a.run = plan.run;
    a.ho_state = reinterpret_cast<float*>(ws + h.state);
    a.ho_flag = reinterpret_cast<unsigned*>(ws + h.flags) + (size_t)pass * plan.blocks * 8;
}
struct BwdSpace {
    Segs fwd, rev;
    Handoff ho;
    size_t qdq, kdk, ck, ends, part, bytes;
};
inline BwdSpace carve_bwd(const Problem& p, const Plan& plan) {
    Carve c;
    BwdSpace b;
    b.fwd = carve_segs(c, p, plan);
    b.rev = carve_segs(c, p, plan);
    b.ho = carve_handoff(c, p, plan, 3);
    const size_t dots = (size_t)p.rows() * p.slabs() * sizeof(float);
    const size_t units = (size_t)p.geom.slots(p.ck_every()) * p.geom.H;
    b.qdq = c.take(dots);
    b.kdk = c.take(dots);
    b.ck = c.take(units * p.D * p.D * sizeof(float));
    b.ends = c.take(units * p.ends() * sizeof(float));
    b.part = c.take(units * sizeof(float));
    b.bytes = c.at;
    return b;
}
inline size_t fwd_workspace(const Problem& p) {
    Carve c;
    const Plan plan = make_plan(p);
    (void)carve_segs(c, p, plan);
    (void)carve_handoff(c, p, plan, 1);
    return c.at;
}
inline size_t bwd_workspace(const Problem& p) { return carve_bwd(p, make_plan(p)).bytes; }

template <typename Tin, bool kRev, bool kStateOnly>
inline cudaError_t run_pass(const Pass<Tin>& a, const Problem& p, cudaStream_t stream) {
    if constexpr (sizeof(Tin) == 2) {
        // (without a token there are no tensors to map: only states are copied)
        if (p.chunked && p.geom.T > 0)
            return tc::launch_pass<kRev, kStateOnly>(a, p.B, p.D, stream);
    }
    return launch_recurrent_pass<Tin, kRev, kStateOnly>(a, p.D, stream);
}

// The states before every segment, from y, z and the states before the first token.
template <typename Tin, bool kRev>
inline cudaError_t run_segments(Pass<Tin> a, const Problem& p, const float* init, uint8_t* ws,
                                const Segs& s, cudaStream_t stream) {
    a.seg_state = reinterpret_cast<float*>(ws + s.state);
    a.seg_decay = reinterpret_cast<float*>(ws + s.decay);
    if (const cudaError_t e = run_pass<Tin, kRev, true>(a, p, stream); e != cudaSuccess) return e;
    const long long n = (long long)p.geom.N * p.geom.H * (p.D * p.D / 4);
    if ((n + 255) / 256 > 0x7fffffffLL) return cudaErrorInvalidValue;
    la_chain_kernel<kRev><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(
        p.geom, init, a.seg_state, a.seg_decay, a.seg, p.D * p.D);
    return cudaGetLastError();
}

template <typename Tin>
inline cudaError_t forward(const Problem& p, const Tin* q, const Tin* k, const Tin* v, const Tin* g,
                           int g_per_head, const float* s0, const uint8_t* mask, Tin* o, float* sT,
                           float scale, uint8_t* ws, cudaStream_t stream) {
    const Plan plan = make_plan(p);
    Carve c;
    const Segs s = carve_segs(c, p, plan);
    const Handoff ho = carve_handoff(c, p, plan, 1);
    Pass<Tin> a{};
    a.geom = p.geom;
    a.wait_ns = p.wait_ns;
    a.handoff_at_once = p.handoff_at_once;
    a.x = q;
    a.y = k;
    a.z = v;
    a.g = g;
    a.g_per_head = g_per_head;
    a.mask = mask;
    a.out = o;
    a.pair_scale = a.inter_scale = scale;
    a.key_scale = 1.f;
    a.parts = sT || plan.split ? 3 : 2;
    a.seg = plan.seg;
    a.init = s0;
    a.fin = sT;
    if (plan.run > 0 && p.geom.T > 0) {
        if (const cudaError_t e = cudaMemsetAsync(ws + ho.flags, 0, ho.flag_bytes, stream);
            e != cudaSuccess)
            return e;
        use_handoff(a, plan, ho, ws, 0);
    }
    if (plan.split) {
        if (const cudaError_t e = run_segments<Tin, false>(a, p, s0, ws, s, stream);
            e != cudaSuccess)
            return e;
        a.init = reinterpret_cast<float*>(ws + s.state);
        a.init_by_slot = 1;
    }
    return run_pass<Tin, false, false>(a, p, stream);
}

template <typename Tin>
inline cudaError_t backward(const Problem& p, const Tin* q, const Tin* k, const Tin* v,
                            const Tin* g, int g_per_head, const float* s0, const uint8_t* mask,
                            const Tin* dout, const float* dsT, Tin* dq, Tin* dk, Tin* dv, Tin* dg,
                            float* ds0, float scale, uint8_t* ws, cudaStream_t stream) {
    const Plan plan = make_plan(p);
    const BwdSpace b = carve_bwd(p, plan);
    Pass<Tin> f{};  // in the direction of time: dq = A(do, v, k), state S^T
    f.geom = p.geom;
    f.wait_ns = p.wait_ns;
    f.handoff_at_once = p.handoff_at_once;
    f.g = g;
    f.g_per_head = g_per_head;
    f.mask = mask;
    // (one part would add as much error to dq, dk and dg as all other roundings: 3.6e-3 in dk of
    // a padded batch, two 2.3e-3)
    f.parts = plan.split ? 3 : 2;
    f.seg = plan.seg;
    Pass<Tin> r = f;  // against it
    r.pair_scale = r.key_scale = scale;
    r.inter_scale = 1.f;
    r.parts = ds0 || plan.split ? 3 : 2;
    f.pair_scale = f.inter_scale = scale;
    f.key_scale = 1.f;
    f.init = s0;
    r.init = dsT;
    if (plan.split) {
        Pass<Tin> a = f;
        a.y = k;
        a.z = v;
        a.parts = 3;
        cudaError_t e = run_segments<Tin, false>(a, p, s0, ws, b.fwd, stream);
        if (e != cudaSuccess) return e;
        a = r;
        a.y = q;
        a.z = dout;
        e = run_segments<Tin, true>(a, p, dsT, ws, b.rev, stream);
        if (e != cudaSuccess) return e;
        f.init = reinterpret_cast<float*>(ws + b.fwd.state);
        r.init = reinterpret_cast<float*>(ws + b.rev.state);
        f.init_by_slot = r.init_by_slot = 1;
    }
    const bool runs = plan.run > 0 && p.geom.T > 0;
    if (runs) {
        const cudaError_t e = cudaMemsetAsync(ws + b.ho.flags, 0, b.ho.flag_bytes, stream);
        if (e != cudaSuccess) return e;
        use_handoff(f, plan, b.ho, ws, 0);
        use_handoff(r, plan, b.ho, ws, 1);
    }
    f.x = dout;
    f.y = v;
    f.z = k;
    f.out = dq;
    f.init_transposed = 1;
    f.dots_stride = r.dots_stride = p.rows();
    if (dg) {
        f.dot_with = q;
        f.dots = reinterpret_cast<float*>(ws + b.qdq);
        f.ck = ws + b.ck;
    }
    cudaError_t e = run_pass<Tin, false, false>(f, p, stream);
    if (e != cudaSuccess) return e;
    Pass<Tin> a = r;  // dv = A'(k, q, do), state G
    a.x = k;
    a.y = q;
    a.z = dout;
    a.out = dv;
    a.fin = ds0;
    if (e = run_pass<Tin, true, false>(a, p, stream); e != cudaSuccess) return e;
    a = r;  // dk = A'(v, do, q), state G^T
    if (runs) use_handoff(a, plan, b.ho, ws, 2);
    a.x = v;
    a.y = dout;
    a.z = q;
    a.parts = 2;  // its state is no result
    a.out = dk;
    a.init_transposed = 1;
    if (dg) {
        a.dot_with = k;
        a.dots = reinterpret_cast<float*>(ws + b.kdk);
        a.ck = ws + b.ck;
        a.ck_dot = reinterpret_cast<float*>(ws + b.ends);
    }
    if (e = run_pass<Tin, true, false>(a, p, stream); e != cudaSuccess) return e;
    if (!dg) return cudaSuccess;
    const long long slots = p.geom.slots(p.ck_every()), warps = slots * p.geom.H;
    float* part = reinterpret_cast<float*>(ws + b.part);
    auto dg_kernel = p.chunked ? la_dg_kernel<Tin, kChunk> : la_dg_kernel<Tin, kRecChunk>;
    dg_kernel<<<(unsigned)((warps + 3) / 4), 128, 0, stream>>>(
        p.geom, mask, f.dots, a.dots, p.slabs(), p.rows(), a.ck_dot, p.ends(),
        g_per_head ? nullptr : dg,
        g_per_head ? part : nullptr);
    if (e = cudaGetLastError(); e != cudaSuccess || !g_per_head) return e;
    la_dg_sum_kernel<Tin><<<p.geom.H, 256, 0, stream>>>(p.geom, part, slots, dg);
    return cudaGetLastError();
}

}  // namespace la
}  // namespace wkv7
