// la_chunked.cuh -- one pass of the decay linear attention on tcgen05 tensor cores, in
// chunks of 128 tokens: bf16, head sizes 64 and 128, forward and backward in time.
//
// With c_t the prefix sums of the log decays inside the chunk, U0 the state before the chunk
// (in the pass's direction), E_ts = e^{c_t - c_s} for s <= t (backward in time: e^{c_s - c_t}
// for s >= t), f_t = e^{c_t} (e^{c_L - c_t}) and k_s = e^{c_L - c_s} (e^{c_s}):
//     out = f . (X U0) + (E . X Y^T) Z,        U1 = e^{c_L} U0 + (k . Y)^T Z
// Four products per chunk:
//     P  = X Y^T   (128 x 128, contraction D)      then E, the mask and the scale -> bf16
//     Oi = P Z     (128 x D, contraction 128)      P read from tensor memory
//     Ox = X U0    (128 x D, contraction D)        U0 rounded to bf16
//     dU = (k . Y)^T Z   (D x D, contraction 128, once for each bf16 part of k . Y)
// Every exponent is a difference over a stretch of tokens, so decays need no bound (nothing is
// divided by a small prefix).  Inside a 32-token block it is a difference of two prefix sums of
// the chunk, off by their half steps: 1e-5 of E with ordinary decays, up to 0.4 % (bf16's own half
// step) behind 100 resets in the same chunk.  X, Y, Z enter raw, as TMA left them.
//
// Roundings to bf16: P (as the scores of any attention) and the copy of U0 that Ox reads, each a half
// step of bf16 of one of the two terms of out.  The state itself is fp32 in registers, and where it
// is a result (a final state, dS0, a segment's start) its update's operand is split in three
// bf16 parts (24 bits), so that it is as good as fp32's: 7e-7 off at most (1.1e-6 in a head whose
// memory is 4096 tokens), with two parts 2.5e-6, with one 2e-3.  Where it only makes bf16 results
// two parts do.  In all o and the gradients are 2.34e-3 off in the 2-norm, rounded once 1.66e-3.
//
// What bounds it.  At D = 64 a chunk moves 64 KB from and to HBM (1.5 us at an SM's even share)
// and takes about 1400 cycles of MMA; it takes 2.4 us, because the roles of a chunk
// (below) each run on one warp per scheduler, at a third of its issue rate: latencies of
// tensor memory, shared memory and barriers, and instruction fetch (see wait_slow).  At D = 128
// it takes 4.6 us against 3 us.
// B = 8, T = 4096, H = 64 of 64: 310 to 336 us from GPU to GPU, 3.3 to 3.5 TB/s, half of the
// measured copy rate (the recurrence 4.75 ms); 16384 tokens of 16 heads of 128: 137 us with its
// states made beforehand.  The gradients' passes at the first: 296 us (dv), 440 us (dq, with
// states kept), 500 us (dk).  All of these move by some percent with where the roles' code falls
// (310 to 320 and 1250 to 1340 us for forward and backward between builds that differ in cold
// code only), so small changes want both timed.
// Tried and left: output staged in a tile of its own (the smaller ring cost as much); rows
// of the decay scan on all lanes (slower: longer shuffles); waits as calls (each cost the MMA
// warp 200 cycles more); score blocks of 32 columns (faster alone, slower with all SMs at it).
//
// One persistent CTA of 16 warps per SM, each with one job, so that a chunk's dependent steps
// overlap with other chunks':
//     warp 0       TMA loads of X, Y, Z into a ring of stages (3 at D = 64, 2 at D = 128)
//     warp 1       issues all MMAs
//     warp 2       decays: prefix sums, factors; clears Z's unused rows
//     warp 3       output tiles shared -> HBM, frees the stage's Z
//     warps 4-7    P: scores -> E . scores in bf16, in place in tensor memory;
//                  at D = 128 also half of k . Y
//     warps 8-11   half of k . Y in parts; the state (at D = 128 half its columns)
//     warps 12-15  out = f . Ox + Oi; at D = 64 the other half of k . Y, at D = 128 the other
//                  half of the state
// The chain from one chunk to the next is only U0 -> bf16 -> Ox and (D = 128) dU -> U1; the state
// never goes through tensor memory.  All waits are on mbarriers (or a flag in global memory)
// and bounded; a thread that gives up sets a flag that ends every other wait, so the CTA
// always reaches its end, waits for its copies and MMAs in flight (bounded), frees its tensor
// memory and reports WKV7_ERR_DEVICE_TIMEOUT (tests/test_linear_attention_timeout.py).
#pragma once
#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "chunked.cuh"
#include "f32x2.cuh"
#include "la_common.cuh"
#include "sm100.cuh"

namespace wkv7 {
namespace la {
namespace tc {

using namespace sm100;

constexpr int kThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
    static constexpr int kStages = D == 64 ? 3 : 2;
    static constexpr int kSub = 128 * 128;            // 128 rows of 64 bf16
    static constexpr int kTile = (D / 64) * kSub;     // an X, Y, Z or output tile
    static constexpr int kStage = 3 * kTile;
    static constexpr int kStateSub = D * 128;         // D rows of 64 bf16
    static constexpr int kStateBytes = (D / 64) * kStateSub;
    // D = 64: k . Y is made a chunk ahead, its second and third part in tiles of their own (two
    // sets), and P and dU are double in tensor memory, so that only the state itself ties a
    // chunk to the next.  D = 128 has room for neither: the parts lie over X and over U0's
    // copy once their products are done.
    static constexpr bool kAhead = D == 64;
    static constexpr bool kPartsInPlace = !kAhead;
    static constexpr int kStateWarps = D == 64 ? 4 : 8;
    static constexpr int OFF_STATE = kStages * kStage;
    static constexpr int OFF_PARTS = OFF_STATE + kStateBytes;
    static constexpr int OFF_SC = OFF_PARTS + (kPartsInPlace ? 0 : 4 * kTile);
    static constexpr int kScBytes = 2 * 512 + 64;     // struct Scan
    // Slots of decays: with two for each stage, a slot is used again only when a chunk that
    // came after all its readers' work is done (one for each stage where there is no room:
    // free with the stage's Z, behind the output).
    static constexpr int kScans = kAhead ? 2 * kStages : kStages;
    static constexpr int OFF_BAR = OFF_SC + kScans * kScBytes;
    static constexpr int kBytes = OFF_BAR + 352;
    // tensor memory columns
    static constexpr int TM_P = 0, TM_OI = kAhead ? 256 : 128, TM_OX = TM_OI + D, TM_DU = TM_OX + D;
};

// One stage's decays.  Tokens come in blocks of 32; a block's border is its last token
// (backward in time: its first), the nearest to the tokens that its keys reach.
struct Scan {
    float c[128];      // prefix sums of log2 decays
    float f[128];      // from the token to its block's border; 0 for tokens that do not enter
    float kb[4];       // key_scale * from the block's border to the chunk's end: k_s = f kb
    uint32_t live[4];  // tokens that enter as keys
    uint32_t out[4];   // rows that get an output (others are written as 0)
    float decay;       // e^{c_L}
    int more;          // another chunk follows in this CTA
    float pad[2];
};
static_assert(sizeof(Scan) == 1088, "kScBytes");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
// The bf16 pair of two fp32, and back.
__device__ __forceinline__ uint32_t pack2(uint64_t x) {
    float a, b;
    split2(x, a, b);
    return pack_bf16(a, b);
}
__device__ __forceinline__ uint64_t unpack2(uint32_t x) {
    return pair2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
// 32 lanes x 8 columns of packed bf16 pairs.
__device__ __forceinline__ void tmem_st_raw8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                     taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// Four 8 x 8 blocks of 16-bit pairs, a warp-MMA fragment each, to rows of 16 bytes: lane l gives the
// address of row l % 8 of block l / 8.
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
                 "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}\n" : "=r"(p));
    return p != 0;
}
// D (tensor memory) += A (tensor memory, bf16 pairs, 8 columns per 16 of the contraction) B.
__device__ __forceinline__ void umma_bf16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The CTA's barriers (8 bytes each, from OFF_BAR).
enum Bar {
    kFull = 0,     // [4] a stage's X and Y have landed
    kFullZ = 4,    // [4] a stage's Z has landed
    kEmpty = 8,    // [4] a stage's X and Y may be loaded again
    kEmptyZ = 12,  // [4] a stage's Z may be loaded again
    kScan = 16,    // [6] a chunk's decays are there (and its unused Z rows are clear)
    kScore = 22,   // [2] P = X Y^T is done
    kCross = 24,   // [2] Ox = X U0 is done
    kPReady = 26,  // [2] P in bf16 is in tensor memory
    kKReady = 28,  // [2] k . Y is in shared memory
    kDelta = 30,   // [2] dU is done
    kStore = 32,   // [4] a stage's output tile is in shared memory
    kSReady = 36,  // U0 in bf16 is in shared memory (and the last dU has been read)
    kOut = 37,     // Ox, Oi and every other product of the chunk are done
    kOFree = 38,   // Ox and Oi have been read
    kDrain = 39,   // all MMAs are done
    kBars = 40
};

// The slow path of a wait, out of line: the roles' code has to fit the SM's instruction cache
// together (as unrolled as each role alone would like it did not, and with all SMs at it
// every role ran at the pace of instruction fetches from the level behind, half as fast).
// Polls for at most `limit` ns, or until another thread has given up.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort,
                                       uint64_t limit) {
    uint64_t t0 = 0;
    for (uint32_t k = 0; k < (1u << 28); ++k) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((k & 63u) == 63u) {  // (the timer is slow to read: not before it matters)
            if (*abort) return false;
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > limit) break;
        }
    }
    *abort = 1;
    raise_flag(4 /* WKV7_ERR_DEVICE_TIMEOUT */);
    return false;
}

__device__ __noinline__ bool handoff_slow(const unsigned* flag, volatile int* abort, uint64_t limit) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t k = 0; k < (1u << 28); ++k) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v != 0) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > limit) break;
        __nanosleep(100);
    }
    *abort = 1;
    raise_flag(4 /* WKV7_ERR_DEVICE_TIMEOUT */);
    return false;
}

struct Ctx {
    uint32_t sbase, bars;
    volatile int* abort;
    uint64_t limit;  // of a wait, in ns
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8 * i; }
    // A bounded wait; false: give up (every role then leaves its loop).
    __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
        return mbar_try_wait(bar(i), parity) || wait_slow(bar(i), parity, abort, limit);
    }
    // The same for a whole warp: all lanes go on, or none (what follows is warp-wide).
    __device__ __forceinline__ bool wait_warp(int i, uint32_t parity) const {
        return __all_sync(0xffffffffu, wait(i, parity));
    }
    __device__ __forceinline__ void arrive(int i) const { mbar_arrive(bar(i)); }
    // The flag of a state handed on, for a whole warp (bounded as the other waits).
    __device__ __forceinline__ bool wait_handoff(const unsigned* flag, int at_once) const {
        return __all_sync(0xffffffffu, handoff_slow(flag, abort, at_once ? 0 : limit));
    }
};

// A role's place in the list of chunks: the n-th of the CTA, in stage st for the ph-th time and
// in decay slot sc for the sp-th.
template <int NS, int NC>
struct Place {
    int n = 0, st = 0, sc = 0;
    uint32_t ph = 0, sp = 0;
    __device__ __forceinline__ void next() {
        ++n;
        if (++st == NS) {
            st = 0;
            ph ^= 1;
        }
        if (++sc == NC) {
            sc = 0;
            sp ^= 1;
        }
    }
    __device__ __forceinline__ uint32_t odd() const { return n & 1; }          // one barrier
    __device__ __forceinline__ uint32_t pair() const { return (n >> 1) & 1; }  // two in turn
};

// Schedule: which chunks a CTA works on, as pieces (consecutive chunks of one (sequence,
// head)); every role walks the same list.
//  - Segments (run == 0): the sequences' segments round robin.  For few (sequence, head)
//    pairs, whose segments start from states made beforehand, and for passes over states only.
//  - Runs: all chunks, laid end to end (heads, sequences, chunks in the direction of the
//    pass), are cut into equal runs, one per CTA, and a CTA takes its run's pieces from the
//    last to the first.  A sequence cut between CTAs m and m + 1 thus has its first chunks
//    at the start of m's work and its last ones at the end of m + 1's: the state that m hands
//    on (through ho_state[m]) is there long before it is needed, unless a sequence is
//    longer than a run.  A CTA only ever waits for the one before it, so the order in which
//    blocks start is enough for progress.
// Without runs 512 sequences of one length on 148 SMs take 4 rounds for 3.46 rounds' work.
// (Slot and chunk numbers fit 32 bits: the entry points check.)
struct Piece {
    Item it;
    int h, slot, tb, te, chunks;  // tokens [tb, te) of the sequence
    bool begins, ends;            // its first (last) chunk in the direction of the pass is the sequence's
};
struct Cursor {
    int item, items;  // segments; or positions: the next one, the run's first
    int slots;        // of the chunks (runs), 0: segments
};
// Blocks that share the segments; on the host, where a test walks them, one has them all.  (As a
// number in the cursor it cost the gradients' kernels 40 to 80 bytes of spills.)
__host__ __device__ __forceinline__ int grid_blocks() {
#ifdef __CUDA_ARCH__
    return (int)gridDim.x;
#else
    return 1;
#endif
}
// Where a block begins.
__host__ __device__ __forceinline__ Cursor first_cursor(const Geom& g, int seg, int run, int block) {
    Cursor at;
    if (run == 0) {
        at.slots = 0;
        at.item = block - grid_blocks();
        at.items = (int)(g.slots(seg) * g.H);
    } else {
        at.slots = (int)g.slots(kChunk);
        const long long all = (long long)at.slots * g.H, start = (long long)block * run;
        at.items = (int)start;
        at.item = (int)(start + run < all ? start + run : all) - 1;
    }
    return at;
}
// The cursor's next piece; chunks < 0: none left.  Out of line: divisions, in every role.
__host__ __device__ __noinline__ Piece next_piece(const Geom& g, int seg, Cursor& at, int rev, int state_only) {
    Piece s;
    s.tb = s.te = 0;
    s.chunks = -1;
    s.begins = s.ends = false;
    if (at.slots == 0) {
        while (at.items - at.item > grid_blocks()) {
            at.item += grid_blocks();
            s.slot = at.item / g.H;
            s.h = at.item - s.slot * g.H;
            s.it = locate(g, s.slot, seg);
            if (s.it.n < 0) continue;
            s.begins = rev ? s.it.j == s.it.nseg - 1 : s.it.j == 0;
            s.ends = rev ? s.it.j == 0 : s.it.j == s.it.nseg - 1;
            if (state_only && s.ends) continue;  // (its state starts no other segment)
            s.tb = s.it.j * seg;
            s.te = s.it.len - s.tb < seg ? s.it.len : s.tb + seg;
            s.chunks = (s.te - s.tb + kChunk - 1) / kChunk;
            return s;
        }
        return s;
    }
    while (at.item >= at.items) {
        const int pos = at.item;
        s.h = pos / at.slots;
        const int in_head = pos - s.h * at.slots;
        s.slot = rev ? at.slots - 1 - in_head : in_head;
        s.it = locate(g, s.slot, kChunk);
        if (s.it.n < 0) {
            --at.item;
            continue;
        }
        const int total = s.it.nseg;  // chunks [first, last] in the direction of the pass
        const int last = rev ? total - 1 - s.it.j : s.it.j;
        const int first = last - (pos - at.items) > 0 ? last - (pos - at.items) : 0;
        s.begins = first == 0;
        s.ends = last == total - 1;
        s.tb = kChunk * (rev ? total - 1 - last : first);
        const int te = kChunk * (rev ? total - first : last + 1);
        s.te = s.it.len < te ? s.it.len : te;
        s.chunks = (s.te - s.tb + kChunk - 1) / kChunk;
        at.item = pos - (last - first + 1);
        return s;
    }
    return s;
}
template <bool kRev, bool kStateOnly>
struct Walk : Piece {
    Cursor at;
    template <typename P>
    __device__ __forceinline__ explicit Walk(const P& p)
        : at(first_cursor(p.geom, p.seg, kStateOnly ? 0 : p.run, (int)blockIdx.x)) {}
    // The next piece; false: none left.
    template <typename P>
    __device__ __forceinline__ bool next(const P& p) {
        Cursor c = at;
        static_cast<Piece&>(*this) = next_piece(p.geom, p.seg, c, kRev, kStateOnly);
        at = c;
        return this->chunks >= 0;
    }
    __device__ __forceinline__ int first_token(int i) const {
        return this->tb + kChunk * (kRev ? this->chunks - 1 - i : i);
    }
    // Number of the chunk that starts at token t0 (128-token slots of all sequences) and head.
    __device__ __forceinline__ long long unit(const Geom& g, int t0) const {
        const int c = t0 / kChunk;
        const int slot = g.cu ? this->it.bos / kChunk + this->it.n + c
                              : this->it.n * Geom::segs(g.T, kChunk) + c;
        return (long long)slot * g.H + this->h;
    }
};

// k . Y for `turns` x 128 groups of 8 elements from group `first` of a 128 x 64 tile, in `parts`
// bf16 parts (the first in place).  Out of line: one copy for the warps that share it.
__device__ __noinline__ void split_keys(uint32_t y, uint32_t part1, uint32_t part2, const Scan* sc,
                                        int first, int turns, int parts) {
    const uint64_t minus = pair2(-1.f, -1.f);
#pragma unroll 1
    for (int u = 0; u < turns; u += 2) {
        uint64_t a[2][4];
        uint32_t w[2][4], at[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int idx = first + (u + h) * 128 + (threadIdx.x & 127), row = idx >> 3;
            at[h] = idx * 16;
            const float f = sc->f[row] * sc->kb[row >> 5];
            uint4 v = ld_shared16(y + at[h]);
            if (f == 0.f) v = make_uint4(0, 0, 0, 0);  // whatever the row holds
            const uint64_t ff = pair2(f, f);
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                a[h][q] = mul2(unpack2(in[q]), ff);
                w[h][q] = pack2(a[h][q]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            st_shared16(y + at[h], w[h][0], w[h][1], w[h][2], w[h][3]);
        if (parts > 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[h][q] = fma2(unpack2(w[h][q]), minus, a[h][q]);
                    w[h][q] = pack2(a[h][q]);
                }
                st_shared16(part1 + at[h], w[h][0], w[h][1], w[h][2], w[h][3]);
            }
        }
        if (parts > 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[h][q] = pack2(fma2(unpack2(w[h][q]), minus, a[h][q]));
                st_shared16(part2 + at[h], w[h][0], w[h][1], w[h][2], w[h][3]);
            }
        }
    }
}

// TMA coordinates (1, 2) of the row of token t.
struct At {
    int c1, c2;
};
__device__ __forceinline__ At tma_row(const Geom& g, const Item& it, int h, int t) {
    if (g.head_first) return {it.bos + t, it.bb * g.H + h};
    return {h, it.bb * g.T + it.bos + t};
}

// kGrad: for dg (states kept or met, dot products of outputs).
template <int D, bool kRev, bool kStateOnly, bool kGrad>
__global__ void __launch_bounds__(kThreads, 1)
la_chunked_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
                  const __grid_constant__ CUtensorMap tm_z,
                  const __grid_constant__ CUtensorMap tm_out,
                  const __grid_constant__ Pass<__nv_bfloat16> p) {
    using C = Cfg<D>;
    constexpr int NS = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Geom& G = p.geom;
    if (!seqlens_ok(G, tid, kThreads)) {
        if (tid == 0 && blockIdx.x == 0) raise_flag(5 /* WKV7_ERR_DEVICE_BAD_SEQLENS */);
        return;
    }
    Ctx cx;
    cx.sbase = smem_u32(smem);
    cx.bars = cx.sbase + C::OFF_BAR;
    // A second (wait_ns); and for a sequence longer than a run, the CTAs before this one work on it in turn
    // first (20 us for each of their chunks, several times what one takes).
    cx.limit = p.wait_ns + 20000ull * (uint64_t)p.run * blockIdx.x;
    cx.abort = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 8 * kBars);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8 * kBars + 4);
    if (cx.sbase & 1023u) {  // the swizzled tiles need a 1024-byte aligned base
        if (tid == 0) raise_flag(3 /* WKV7_ERR_CUDA */);
        return;
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    if (tid == 32) {
        *cx.abort = 0;
        for (int i = 0; i < kBars; ++i) {
            const int count = i >= kEmptyZ && i < kEmptyZ + 4 ? (kStateOnly ? 32 * C::kStateWarps : 1)
                              : i >= kStore && i < kStore + 4 ? 128
                              : i == kPReady || i == kPReady + 1 || i == kOFree ? 128
                              : i == kKReady || i == kKReady + 1 ? 256
                              : i == kSReady ? 32 * C::kStateWarps
                                             : 1;
            mbar_init(cx.bar(i), count);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    auto scan_of = [&](int sc) {
        return reinterpret_cast<Scan*>(smem + C::OFF_SC + sc * C::kScBytes);
    };
    Walk<kRev, kStateOnly> wk(p);
    using Spot = Place<NS, C::kScans>;
    Spot at_;
    int& n = at_.n;

    // A chunk's output is staged over its Z once all its products are done (Z is the tile that
    // the next chunk of the stage needs last; X and Y are loaded again before).
    auto out_tile = [&](const Spot& at) { return cx.sbase + at.st * C::kStage + 2 * C::kTile; };
    // k . Y of one chunk, in bf16 parts: the first over Y itself.  Two groups of four warps take
    // half of it each: of the rows at D = 64, of the columns at D = 128.
    auto scale_keys = [&](const Spot& at, int half) {
        const int st = at.st;
        if (!cx.wait_warp(kScan + at.sc, at.sp)) return false;
        if (!cx.wait_warp(kFull + st, at.ph)) return false;
        if (!kStateOnly && !cx.wait_warp(kScore + (at.n & 1), at.pair())) return false;
        if (C::kPartsInPlace) {
            // X and U0's copy have been read; without them, the last chunk's parts
            if (!kStateOnly && !cx.wait_warp(kCross + (at.n & 1), at.pair())) return false;
            if (kStateOnly && at.n > 0 &&
                !cx.wait_warp(kDelta + ((at.n - 1) & 1), ((at.n - 1) >> 1) & 1))
                return false;
        }
        const uint32_t x = cx.sbase + st * C::kStage, y = x + C::kTile;
        const uint32_t part1 =
            C::kPartsInPlace ? x : cx.sbase + C::OFF_PARTS + 2 * C::kTile * (at.n & 1);
        const uint32_t part2 = C::kPartsInPlace ? cx.sbase + C::OFF_STATE : part1 + C::kTile;
        const uint32_t o = D == 64 ? 0 : half * C::kSub;
        split_keys(y + o, part1 + o, part2 + o, scan_of(at.sc), D == 64 ? half * 512 : 0, D / 16,
                   p.parts);
        fence_proxy_async();
        cx.arrive(kKReady + (at.n & 1));
        return true;
    };

    // ------------------------------------------------------------------ warp 0: loads
    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int z_loads = 0;
            while (ok && wk.next(p)) {
                for (int i = 0; ok && i < wk.chunks; ++i, at_.next()) {
                    const int st = at_.st;
                    if (n >= NS && !(ok = cx.wait(kEmpty + st, at_.ph ^ 1))) break;
                    const uint32_t full = cx.bar(kFull + st), at = cx.sbase + st * C::kStage;
                    const uint32_t fz = cx.bar(kFullZ + st);
                    mbar_arrive_expect_tx(full, (kStateOnly ? 1 : 2) * C::kTile);
                    const At a = tma_row(G, wk.it, wk.h, wk.first_token(i));
#pragma unroll
                    for (int s = 0; s < D / 64; ++s) {
                        if (!kStateOnly)
                            tma_load_3d(at + s * C::kSub, &tm_x, full, 64 * s, a.c1, a.c2);
                        tma_load_3d(at + C::kTile + s * C::kSub, &tm_y, full, 64 * s, a.c1, a.c2);
                    }
                    if (n >= NS && !(ok = cx.wait(kEmptyZ + st, at_.ph ^ 1))) {
                        at_.next();  // (for the drain below)
                        break;
                    }
                    mbar_arrive_expect_tx(fz, C::kTile);
#pragma unroll
                    for (int s = 0; s < D / 64; ++s)
                        tma_load_3d(at + 2 * C::kTile + s * C::kSub, &tm_z, fz, 64 * s, a.c1, a.c2);
                    z_loads = n + 1;
                }
            }
            // The copies in flight land before the CTA leaves (bounded), also when this role is
            // done and another gives up.
            for (int m = n < NS ? 0 : n - NS; m < n; ++m)
                (void)mbar_wait(cx.bar(kFull + m % NS), (m / NS) & 1);
            for (int m = z_loads < NS ? 0 : z_loads - NS; m < z_loads; ++m)
                (void)mbar_wait(cx.bar(kFullZ + m % NS), (m / NS) & 1);
        }
    }
    // ------------------------------------------------------------------ warp 1: MMAs
    else if (warp == 1) {
        {
            // The whole warp walks the list, so that descriptors stay in uniform registers (an
            // MMA takes its operands from there); one elected lane issues.
            const bool leader = elect_one();
            const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
            bool ok = true;
            constexpr uint32_t id_score = idesc_bf16(128, 128, false, false);
            constexpr uint32_t id_out = idesc_bf16(128, D, false, true);
            constexpr uint32_t id_delta = idesc_bf16(D, D, true, true);
            // descriptors: an address in 16-byte units added to the layout's constants
            const uint64_t kmaj = smem_desc(0, 16, 1024);                  // K-major
            const uint64_t mn_tile = smem_desc(0, C::kSub, 1024);          // MN-major tiles
            const uint64_t mn_state = smem_desc(0, C::kStateSub, 1024);    // MN-major U0
            Spot sc_at;
            auto score = [&]() {  // P = X Y^T of the next chunk
                const int st = sc_at.st, m = sc_at.n;
                if (!cx.wait_warp(kFull + st, sc_at.ph)) return false;
                sc_at.next();
                tc_fence_after();
                uint64_t a = kmaj + ((cx.sbase + st * C::kStage) >> 4), b = a + (C::kTile >> 4);
                const uint32_t tp = tmem + C::TM_P + (C::kAhead ? 128 * (m & 1) : 0);
#pragma unroll 1
                for (int s = 0; s < D / 64; ++s) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (leader) umma_bf16(tp, a + 2 * kk, b + 2 * kk, id_score, s + kk > 0);
                    a += C::kSub >> 4;
                    b += C::kSub >> 4;
                }
                if (leader) umma_commit(cx.bar(kScore + (m & 1)));
                return true;
            };
            // The products of chunk n, and the score of the one after it (more); n = -1 for the
            // first score alone.
            auto chunk = [&](bool chunk_n, bool more) {
                const int st = at_.st;
                const uint32_t x = (cx.sbase + st * C::kStage) >> 4, y = x + (C::kTile >> 4),
                               z = y + (C::kTile >> 4), state = (cx.sbase + C::OFF_STATE) >> 4;
                auto delta = [&]() {  // dU, from the parts of k . Y
                    if (!cx.wait_warp(kFullZ + st, at_.ph)) return false;
                    if (!cx.wait_warp(kKReady + (n & 1), at_.pair())) return false;
                    tc_fence_after();
                    const uint32_t own =
                        (cx.sbase + C::OFF_PARTS + 2 * C::kTile * (n & 1)) >> 4;
                    const uint32_t td = tmem + C::TM_DU + (C::kAhead ? 64 * (n & 1) : 0);
#pragma unroll 1
                    for (int part = 0; part < p.parts; ++part) {
                        const uint64_t a =
                            mn_tile + (part == 0          ? y
                                       : C::kPartsInPlace ? (part == 1 ? x : state)
                                                          : own + (part - 1) * (C::kTile >> 4));
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            if (leader)
                                umma_bf16(td, a + 128 * kk, mn_tile + z + 128 * kk, id_delta,
                                          part + kk > 0);
                    }
                    if (leader) umma_commit(cx.bar(kDelta + (n & 1)));
                    return true;
                };
                if (C::kAhead && !kStateOnly) {
                    if (more && !score()) return false;
                    if (!chunk_n) return true;
                    if (!delta()) return false;  // (its last user's dU was read before U0 came)
                }
                if (chunk_n && !cx.wait_warp(kSReady, at_.odd())) return false;
                if (!kStateOnly && chunk_n) {
                    if (n > 0 && !cx.wait_warp(kOFree, at_.odd() ^ 1)) return false;
                    tc_fence_after();
                    uint64_t a = kmaj + x, b = mn_state + state;
#pragma unroll 1
                    for (int s = 0; s < D / 64; ++s) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            if (leader)
                                umma_bf16(tmem + C::TM_OX, a + 2 * kk, b + 128 * kk, id_out, s + kk > 0);
                        a += C::kSub >> 4;
                        b += 512;
                    }
                    if (leader) umma_commit(cx.bar(kCross + (n & 1)));
                    if (!cx.wait_warp(kPReady + (n & 1), at_.pair())) return false;
                    // Z, its unused rows clear (where dU is ahead it has waited for both)
                    if (!C::kAhead && !cx.wait_warp(kScan + at_.sc, at_.sp)) return false;
                    if (!C::kAhead && !cx.wait_warp(kFullZ + st, at_.ph)) return false;
                    tc_fence_after();
                    b = mn_tile + z;
                    const uint32_t tp = tmem + C::TM_P + (C::kAhead ? 128 * (n & 1) : 0);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if (leader) umma_bf16_ts(tmem + C::TM_OI, tp + 8 * kk, b + 128 * kk, id_out, kk > 0);
                }
                if (!C::kAhead && !kStateOnly) {
                    if (more && !score()) return false;
                    if (!chunk_n) return true;
                }
                if ((!C::kAhead || kStateOnly) && !delta()) return false;
                if (leader) {  // the chunk's tiles have been read, too
                    umma_commit(cx.bar(kOut));
                    umma_commit(cx.bar(kEmpty + st));
                }
                return true;
            };
            // Chunk m's score goes with the products of chunk m - 1, so the list is walked one
            // chunk ahead of the products.
            bool started = kStateOnly;
            while (ok) {
                bool have = wk.next(p);
                while (have && wk.chunks == 0) have = wk.next(p);
                const int here = have ? __shfl_sync(0xffffffffu, wk.chunks, 0) : (started && !kStateOnly ? 1 : 0);
                if (here == 0) break;
                for (int i = 0; ok && i < here; ++i) {
                    ok = chunk(started, have);
                    if (started) at_.next();
                    started = true;
                }
                if (!have) break;
            }
            // and so do the MMAs
            if (leader) umma_commit(cx.bar(kDrain));
            (void)mbar_wait(cx.bar(kDrain), 0);
        }
    }
    // ------------------------------------------------------------------ warp 2: decays
    else if (warp == 2) {
        bool ok = true;
        auto next_tokens = [&]() {  // the next segment with tokens
            bool have = wk.next(p);
            while (have && wk.chunks == 0) have = wk.next(p);
            return have;
        };
        bool have = next_tokens();
        while (ok && have) {
            const Rows rw = rows_of(G, wk.it, wk.h);
            const uint8_t* mrow = p.mask ? p.mask + (long long)wk.it.bb * G.T + wk.it.bos : nullptr;
            const int te = wk.te, chunks = wk.chunks;
            const float ghead = p.g_per_head ? clamp_log_decay(to_f32(p.g[wk.h])) : 0.f;
            // four tokens a lane; the next chunk's are in flight while this one is scanned
            uint16_t graw[4] = {0, 0, 0, 0};
            uint8_t mraw[4] = {1, 1, 1, 1};
            auto fetch = [&](int t0) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int t = min(t0 + 4 * lane + q, te - 1);
                    if (!p.g_per_head)
                        graw[q] = reinterpret_cast<const uint16_t*>(p.g)[rw.first + t * rw.step];
                    if (mrow) mraw[q] = mrow[t];
                }
            };
            if (chunks > 0) fetch(wk.first_token(0));
            for (int i = 0; ok && i < chunks; ++i, at_.next()) {
                const int st = at_.st, t0 = wk.first_token(i) + 4 * lane;
                // log decays, which tokens exist, which update the state
                float gl[4];
                uint32_t in = 0, upd = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    in |= (t0 + q < te ? 1u : 0u) << q;
                    upd |= (t0 + q < te && mraw[q] ? 1u : 0u) << q;
                    const float x =
                        p.g_per_head ? ghead
                                     : clamp_log_decay(__uint_as_float((uint32_t)graw[q] << 16));
                    gl[q] = (upd >> q) & 1 ? x : 0.f;
                }
                if (i + 1 < chunks)
                    fetch(wk.first_token(i + 1));
                else
                    have = next_tokens();
                const uint32_t enter = kRev ? in : upd, outs = kRev ? upd : in;
                // Sums inside a 32-token block (8 lanes): `far` from the token to its border
                // (the tokens after it; backward in time the ones from the block's second
                // to it), summed in that direction, so that it is as exact as it is
                // small; and inclusive prefix sums c.
                const float own = (gl[0] + gl[1]) + (gl[2] + gl[3]);
                float pre = own, far_l = kRev ? ((lane & 7) == 0 ? (gl[1] + gl[2]) + gl[3] : own) : own;
#pragma unroll
                for (int m = 1; m < 8; m <<= 1) {
                    const float a = __shfl_up_sync(0xffffffffu, pre, m, 8);
                    const float b = kRev ? __shfl_up_sync(0xffffffffu, far_l, m, 8)
                                         : __shfl_down_sync(0xffffffffu, far_l, m, 8);
                    if ((lane & 7) >= m) pre += a;
                    if (kRev ? (lane & 7) >= m : (lane & 7) + m < 8) far_l += b;
                }
                // what lies beyond this lane's four tokens
                float far_o = kRev ? __shfl_up_sync(0xffffffffu, far_l, 1, 8)
                                   : __shfl_down_sync(0xffffffffu, far_l, 1, 8);
                if (kRev ? (lane & 7) == 0 : (lane & 7) == 7) far_o = 0.f;
                const float t0s = __shfl_sync(0xffffffffu, pre, 7), t1s = __shfl_sync(0xffffffffu, pre, 15),
                            t2s = __shfl_sync(0xffffffffu, pre, 23), t3s = __shfl_sync(0xffffffffu, pre, 31);
                const int blk = lane >> 3;
                const float before = blk == 0 ? 0.f : blk == 1 ? t0s : blk == 2 ? t0s + t1s : t0s + t1s + t2s;
                const float after = blk == 3 ? 0.f : blk == 2 ? t3s : blk == 1 ? t2s + t3s : t1s + t2s + t3s;
                float c = before + (pre - own);
                float cc[4], ff[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    c += gl[q];
                    cc[q] = c * kLog2e;
                }
                float d = far_o;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int q = kRev ? u : 3 - u;
                    if (kRev && !((lane & 7) == 0 && q == 0)) d += gl[q];
                    ff[q] = (enter >> q) & 1 ? ex2(d * kLog2e) : 0.f;
                    if (!kRev) d += gl[q];
                }
                const float tail = __shfl_sync(0xffffffffu, gl[0], lane & 24);  // rev: the border's own
                if (n >= NS &&
                    !(ok = cx.wait_warp((C::kAhead ? kEmpty : kEmptyZ) + st, at_.ph ^ 1)))
                    break;
                Scan* sc = scan_of(at_.sc);
                *reinterpret_cast<float4*>(&sc->c[4 * lane]) = make_float4(cc[0], cc[1], cc[2], cc[3]);
                *reinterpret_cast<float4*>(&sc->f[4 * lane]) = make_float4(ff[0], ff[1], ff[2], ff[3]);
                // 8 lanes make a 32-token word
                uint32_t lw = enter << (4 * (lane & 7)), ow = outs << (4 * (lane & 7));
#pragma unroll
                for (int m = 1; m < 8; m <<= 1) {
                    lw |= __shfl_xor_sync(0xffffffffu, lw, m);
                    ow |= __shfl_xor_sync(0xffffffffu, ow, m);
                }
                if ((lane & 7) == 0) {
                    sc->live[blk] = lw;
                    sc->out[blk] = ow;
                    sc->kb[blk] = p.key_scale * ex2(kLog2e * (kRev ? before + tail : after));
                }
                // A weak decay's rounding repeats at every chunk that a state lives through: 1 +
                // the small difference, off by half a step of a number near 1 (2^-25; expf's
                // steps are up to four times that).  A strong one is e^sum itself: the
                // difference would be -1 rounded, off by 2^-25 of 1 and not of e^sum (7e-3
                // of it at a sum of -12.8).
                if (lane == 0) {
                    sc->more = i + 1 < chunks || have;
                    const float sum = (t0s + t1s) + (t2s + t3s);
                    sc->decay = fabsf(sum) < 0.5f ? 1.f + expm1f(sum) : expf(sum);
                }
                // rows of Z that do not enter may hold anything (0 * NaN is NaN): clear them
                if (__any_sync(0xffffffffu, enter != 15u)) {
                    if (!(ok = cx.wait_warp(kFullZ + st, at_.ph))) break;
                    const uint32_t z = cx.sbase + st * C::kStage + 2 * C::kTile;
                    for (int q = 0; q < 4; ++q) {
                        if ((enter >> q) & 1) continue;
                        for (int e = 0; e < (D / 64) * 8; ++e)
                            st_shared16(z + (e >> 3) * C::kSub + (4 * lane + q) * 128 + (e & 7) * 16, 0,
                                        0, 0, 0);
                    }
                    fence_proxy_async();
                }
                __syncwarp();
                if (lane == 0) cx.arrive(kScan + at_.sc);
            }
        }
    }
    // ------------------------------------------------------------------ warp 3: stores
    else if (warp == 3) {
        if (!kStateOnly) {
            bool ok = true;
            while (ok && wk.next(p)) {
                const Rows rw = rows_of(G, wk.it, wk.h);
                for (int i = 0; ok && i < wk.chunks; ++i, at_.next()) {
                    const int t0 = wk.first_token(i);
                    if (!(ok = cx.wait_warp(kStore + at_.st, at_.ph))) break;
                    const uint32_t tile = out_tile(at_);
                    if (t0 + kChunk <= wk.te) {
                        if (lane == 0) {
                            const At a = tma_row(G, wk.it, wk.h, t0);
#pragma unroll
                            for (int s = 0; s < D / 64; ++s)
                                tma_store_3d(&tm_out, tile + s * C::kSub, 64 * s, a.c1, a.c2);
                            bulk_commit();
                            bulk_wait_read0();
                        }
                    } else {  // the sequence's last rows: those behind it belong to others
                        for (int e = lane; e < (wk.te - t0) * (D / 8); e += 32) {
                            const int row = e / (D / 8), c = e % (D / 8);
                            const uint4 v = ld_shared16(tile + (c / 8) * C::kSub + row * 128 +
                                                        (((c % 8) ^ (row & 7)) << 4));
                            *reinterpret_cast<uint4*>(
                                p.out + (rw.first + (long long)(t0 + row) * rw.step) * D + 8 * c) = v;
                        }
                        fence_proxy_async();  // the stage's next copy comes behind these reads
                    }
                    __syncwarp();
                    if (lane == 0) cx.arrive(kEmptyZ + at_.st);
                }
            }
            if (lane == 0) bulk_wait0();
        }
    }
    // ------------------------------------------------------------------ warps 4-7: P
    else if (warp < 8) {
        bool ok = true;
        const int w = warp & 3, row = 32 * w + lane;
        while ((!kStateOnly || C::kPartsInPlace) && ok && wk.next(p)) {
            for (int i = 0; ok && i < wk.chunks; ++i, at_.next()) {
                const int st = at_.st;
                if (kStateOnly) {
                    ok = scale_keys(at_, 0);
                    continue;
                }
                const uint32_t tp = tmem + ((uint32_t)(32 * w) << 16) + C::TM_P +
                                    (C::kAhead ? 128 * (n & 1) : 0);
                if (!(ok = cx.wait_warp(kScan + at_.sc, at_.sp))) break;
                const Scan* sc = scan_of(at_.sc);
                const float ct = sc->c[row];
                if (!(ok = cx.wait_warp(kScore + (n & 1), at_.pair()))) break;
                tc_fence_after();
                // Loops stay rolled: four roles share the instruction cache of each
                // sub-partition, and one warp running long straight code is fetch-bound.
#pragma unroll 1
                for (int hb = 0; hb < 8; ++hb) {  // 16 columns at a time
                    const int b = hb >> 1, col = 16 * hb;
                    uint32_t out[8];
                    if (kRev ? b < w : b > w) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) out[q] = 0;
                    } else {
                        float v[16];
                        tmem_ld16(tp + col, v);
                        const uint32_t live = sc->live[b];
                        if (b != w && live == 0xffffffffu) {
                            // token to its block's border to this row: both exponents <= 0
                            const float border = sc->c[kRev ? 32 * b : 32 * b + 31];
                            const float r = p.pair_scale * ex2(kRev ? border - ct : ct - border);
                            const uint64_t rr = pair2(r, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int q = 0; q < 16; q += 4) {
                                const ulonglong2 f =
                                    *reinterpret_cast<const ulonglong2*>(&sc->f[col + q]);
                                out[q / 2] = pack2(mul2(mul2(pair2(v[q], v[q + 1]), rr), f.x));
                                out[q / 2 + 1] = pack2(mul2(mul2(pair2(v[q + 2], v[q + 3]), rr), f.y));
                            }
                        } else {
                            // keys that this row may use: live and, on the diagonal block, not
                            // on the wrong side of the row
                            uint32_t use = live;
                            if (b == w) use &= kRev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
                            use >>= col & 16;
                            const uint64_t sign = kRev ? pair2(1.f, 1.f) : pair2(-1.f, -1.f);
                            const uint64_t cc = kRev ? pair2(-ct, -ct) : pair2(ct, ct);
                            const uint64_t ps = pair2(p.pair_scale, p.pair_scale);
                            tmem_ld_wait();
#pragma unroll
                            for (int q = 0; q < 16; q += 2) {
                                const uint64_t c2 = *reinterpret_cast<const uint64_t*>(&sc->c[col + q]);
                                float ea, eb, a, d;
                                split2(fma2(c2, sign, cc), ea, eb);
                                split2(mul2(mul2(pair2(v[q], v[q + 1]), ps), pair2(ex2(ea), ex2(eb))), a,
                                       d);
                                out[q / 2] = pack_bf16((use >> q) & 1 ? a : 0.f,
                                                       (use >> (q + 1)) & 1 ? d : 0.f);
                            }
                        }
                    }
                    // in place: these 8 columns lie over scores that are read already
                    tmem_st_raw8(tp + 8 * hb, out);
                }
                tmem_st_wait();
                tc_fence_before();
                cx.arrive(kPReady + (n & 1));
                if (C::kPartsInPlace) ok = scale_keys(at_, 0);
            }
        }
    }
    // -------------------------------------- warps 8-15: k . Y and state, outputs and state
    else {
      auto role = [&](auto which) {
        constexpr bool first = decltype(which)::value;  // warps 8-11
        bool ok = true;
        const int w = warp & 3, wt = tid & 127;
        constexpr bool kBoth = D == 128;   // warps 12-15 hold state columns 64..127
        constexpr bool has_state = first || kBoth;
        constexpr int R = D == 64 ? 32 : 64;  // state entries per thread
        const int sthread = first ? wt : 128 + wt;
        constexpr int kSThreads = 32 * C::kStateWarps;
        // Entry i of a thread: at D = 64 the MMA fragment layout of an M = 64 accumulator (rows
        // 16 w + lane / 4 and + 8), at D = 128 row 32 w + lane, 64 columns.
        const int srow = kBoth ? 32 * w + lane : 16 * w + lane / 4;
        const int scol = kBoth ? (first ? 0 : 64) : 2 * (lane & 3);
        float S[R];
        const uint32_t state_s = cx.sbase + C::OFF_STATE;
        // entries (2 m, 2 m + 1) at D = 64: row srow + 8 (m & 1), columns scol + 8 (m / 2) ..
        auto entry = [&](int q, int rs, int cs) {  // offset of entry q for row and column strides
            return kBoth ? srow * rs + (scol + q) * cs
                         : (srow + 8 * ((q >> 1) & 1)) * rs + (scol + 8 * (q >> 2) + (q & 1)) * cs;
        };
        auto load_state = [&](const float* s, bool transposed) {
            constexpr int V = kBoth ? 4 : 2;  // neighbouring columns a thread holds
            if (!transposed) {
#pragma unroll
                for (int q = 0; q < R; q += V) {
                    const float* src = s + entry(q, D, 1);
                    if constexpr (kBoth) {
                        const float4 x = *reinterpret_cast<const float4*>(src);
                        S[q] = x.x; S[q + 1] = x.y; S[q + 2] = x.z; S[q + 3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2*>(src);
                        S[q] = x.x; S[q + 1] = x.y;
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < R; ++q) S[q] = s[entry(q, 1, D)];
            }
        };
        auto save_state = [&](float* s) {
#pragma unroll
            for (int q = 0; q < R; q += kBoth ? 4 : 2) {
                float* dst = s + entry(q, D, 1);
                if constexpr (kBoth)
                    *reinterpret_cast<float4*>(dst) = make_float4(S[q], S[q + 1], S[q + 2], S[q + 3]);
                else
                    *reinterpret_cast<float2*>(dst) = make_float2(S[q], S[q + 1]);
            }
        };
        // U0 in bf16, [row][column] with the columns in 64-wide swizzled blocks
        auto publish_state = [&]() {
            if (!kStateOnly) {
                if constexpr (kBoth) {
                    const uint32_t base = state_s + (first ? 0 : C::kStateSub) + srow * 128;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        st_shared16(base + ((q ^ (srow & 7)) << 4),
                                    pack_bf16(S[8 * q], S[8 * q + 1]),
                                    pack_bf16(S[8 * q + 2], S[8 * q + 3]),
                                    pack_bf16(S[8 * q + 4], S[8 * q + 5]),
                                    pack_bf16(S[8 * q + 6], S[8 * q + 7]));
                } else {
                    // blocks (rows 16 w .., columns 8 c ..), (rows + 8, same), (.., next c), ..
                    const int r = 16 * w + (lane & 15);
#pragma unroll
                    for (int c = 0; c < 8; c += 2)
                        stmatrix4(state_s + r * 128 + (((c + (lane >> 4)) ^ (r & 7)) << 4),
                                  pack_bf16(S[4 * c], S[4 * c + 1]), pack_bf16(S[4 * c + 2], S[4 * c + 3]),
                                  pack_bf16(S[4 * c + 4], S[4 * c + 5]),
                                  pack_bf16(S[4 * c + 6], S[4 * c + 7]));
                }
                fence_proxy_async();
            }
            tc_fence_before();
            cx.arrive(kSReady);
        };
        Spot keys;
        float decay = 0.f, next_decay = 0.f;
        int more = 0, next_more = 0;
        while (ok && wk.next(p)) {
            const long long state_at = ((long long)wk.it.n * G.H + wk.h) * D * D;
            const long long seg_at = ((long long)wk.slot * G.H + wk.h) * D * D;
            const Rows rw = rows_of(G, wk.it, wk.h);
            if (has_state) {
                if (!kStateOnly && p.run > 0 && !wk.begins) {  // handed on by the CTA before
                    const int from = (int)blockIdx.x - 1;
                    if (!(ok = cx.wait_handoff(p.ho_flag + 8 * from + (sthread >> 5),
                                               p.handoff_at_once))) break;
                    const float4* src =
                        reinterpret_cast<const float4*>(p.ho_state + (long long)from * D * D) + sthread;
#pragma unroll
                    for (int q = 0; q < R / 4; ++q) {
                        const float4 x = __ldcg(src + q * kSThreads);
                        S[4 * q] = x.x; S[4 * q + 1] = x.y; S[4 * q + 2] = x.z; S[4 * q + 3] = x.w;
                    }
                } else if (!kStateOnly && p.init) {
                    load_state(p.init + (p.init_by_slot ? seg_at : state_at), p.init_transposed);
                } else {
#pragma unroll
                    for (int q = 0; q < R; ++q) S[q] = 0.f;
                }
            }
            float logs = 0.f;
            for (int i = 0; ok && i < wk.chunks; ++i, at_.next()) {
                const int t0 = wk.first_token(i);
                // What the state's warps need of a stage's decays they read before they give
                // that chunk's U0: from then on the stage may be used up and refilled.
                if (!C::kAhead || n == 0) {
                    if (!(ok = cx.wait_warp(kScan + at_.sc, at_.sp))) break;
                    decay = scan_of(at_.sc)->decay;
                    more = scan_of(at_.sc)->more;
                }
                if (has_state && (C::kAhead || i == 0)) publish_state();
                const Scan* sc = scan_of(at_.sc);
                if (kStateOnly && has_state) logs += sc->c[127];
                float rowf = 0.f;
                bool row_out = true;
                if (!kStateOnly && !first) {
                    const int row = 32 * w + lane;
                    rowf = p.inter_scale * ex2(kRev ? sc->c[127] - sc->c[row] : sc->c[row]);
                    row_out = (sc->out[w] >> lane) & 1;
                }
                // What comes from HBM for dg, the chunk's kept state and the rows of out's dot
                // products, is on its way to L2 a chunk ahead (in registers it would have to
                // live across the work below, and did not fit).
                if constexpr (kGrad) {
                    if (i + 1 < wk.chunks) {
                        const int t1 = wk.first_token(i + 1);
                        if (kRev && has_state) {
                            const float* ck = static_cast<const float*>(p.ck) +
                                              wk.unit(G, t1) * (D * D) + (sthread >> 3) * 32;
                            // 32 floats a line: lines (thread / 8), + kSThreads / 8, ..
                            if ((sthread & 7) == 0) {
#pragma unroll
                                for (int l = 0; l < R / 4; ++l)
                                    prefetch_l2(ck + l * kSThreads * 4);
                            }
                        }
                        const int t = t1 + 32 * w + lane;
                        if (!first && t < wk.te) {
                            const __nv_bfloat16* src =
                                p.dot_with + (rw.first + (long long)t * rw.step) * D;
#pragma unroll
                            for (int l = 0; l < D / 64; ++l) prefetch_l2(src + 64 * l);
                        }
                    }
                }
                // k . Y: of the next chunk where there is room for two (half of it here, half
                // there), of this one with warps 4-7 otherwise
                if (C::kAhead) {
                    for (int k = n == 0 ? 0 : 1; ok && k < 1 + (more ? 1 : 0); ++k) {
                        ok = scale_keys(keys, first ? 0 : 1);
                        next_decay = scan_of(keys.sc)->decay;
                        next_more = scan_of(keys.sc)->more;
                        keys.next();
                    }
                } else if (first) {
                    ok = scale_keys(at_, 1);
                }
                if (!ok) break;

                constexpr bool kRowAhead = kGrad && !first && D == 64;
                uint4 wrow[kRowAhead ? D / 8 : 1];
                if constexpr (kRowAhead) {
                    const int t = t0 + 32 * w + lane;
                    if (t < wk.te && row_out) {
                        const uint4* src = reinterpret_cast<const uint4*>(
                            p.dot_with + (rw.first + (long long)t * rw.step) * D);
#pragma unroll
                        for (int u = 0; u < D / 8; ++u) wrow[u] = src[u];
                    }
                }

                // Backward in time: <S_end, G_end> of the chunk, with G_end rounded as the
                // product X U0 reads it.  What tokens s >= t take from it in dL/dc is then
                // the same sum's own terms, and the difference, e^{c_L - c_t} <S_t, G_end>,
                // decays with t as it should (with the exact G_end the rounding of all terms
                // would stay in dg of tokens that G_end no longer reaches).
                if (kGrad && kRev && has_state) {
                    const long long u = wk.unit(G, t0);
                    const float4* ck = static_cast<const float4*>(p.ck) + u * (D * D / 4) + sthread;
                    float4 kept[R / 4];
#pragma unroll
                    for (int q = 0; q < R / 4; ++q) kept[q] = ck[q * kSThreads];
                    float s = 0.f;
#pragma unroll
                    for (int q = 0; q < R / 4; ++q) {
                        const float4 v = kept[q];
                        const uint32_t a = pack_bf16(S[4 * q], S[4 * q + 1]);
                        const uint32_t b = pack_bf16(S[4 * q + 2], S[4 * q + 3]);
                        s = fmaf(v.x, __uint_as_float(a << 16), s);
                        s = fmaf(v.y, __uint_as_float(a & 0xffff0000u), s);
                        s = fmaf(v.z, __uint_as_float(b << 16), s);
                        s = fmaf(v.w, __uint_as_float(b & 0xffff0000u), s);
                    }
#pragma unroll
                    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                    if (lane == 0) p.ck_dot[u * C::kStateWarps + (sthread >> 5)] = s;
                }

                // (without a state here: for the next chunk's parts' sake)
                if (!(ok = cx.wait_warp(kDelta + (n & 1), at_.pair()))) break;
                tc_fence_after();
                if (has_state) {
                    if constexpr (kBoth) {
#pragma unroll
                        for (int q = 0; q < R; q += 16) {
                            float d[16];
                            tmem_ld16(tmem + ((uint32_t)(32 * w) << 16) + C::TM_DU + scol + q, d);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 16; ++u) S[q + u] = fmaf(decay, S[q + u], d[u]);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < R; q += 16) {
                            float d[16];
                            tmem_ld16x32(tmem + ((uint32_t)(32 * w) << 16) + C::TM_DU + 64 * (n & 1) + 2 * q, d);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 16; ++u) S[q + u] = fmaf(decay, S[q + u], d[u]);
                        }
                    }
                    // forward: keep the state at the chunk's end
                    if (kGrad && !kRev) {
                        const long long u = wk.unit(G, t0);
                        float4* ck = static_cast<float4*>(p.ck) + u * (D * D / 4) + sthread;
#pragma unroll
                        for (int q = 0; q < R / 4; ++q)
                            ck[q * kSThreads] =
                                make_float4(S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]);
                    }
                    // the next chunk's U0, once the product that reads this one is done
                    if (C::kAhead && !kStateOnly &&
                        !(ok = cx.wait_warp(kCross + (n & 1), at_.pair())))
                        break;
                    if (!C::kAhead && i + 1 < wk.chunks) publish_state();  // (before any output)
                    if (kStateOnly) cx.arrive(kEmptyZ + at_.st);
                }
                if (C::kAhead) {
                    decay = next_decay;
                    more = next_more;
                }

                if (!kStateOnly && !first) {  // outputs
                    if (!(ok = cx.wait_warp(kOut, at_.odd()))) break;
                    tc_fence_after();
                    const uint32_t tile = out_tile(at_);
                    const int row = 32 * w + lane, t = t0 + row;
                    const bool in = t < wk.te;
                    const long long grow = rw.first + (long long)t * rw.step;
                    const uint32_t to = tmem + ((uint32_t)(32 * w) << 16);
                    float dot = 0.f;
                    constexpr int V = 16;
#pragma unroll 1
                    for (int q = 0; q < D; q += V) {
                        float ox[V], oi[V];
                        tmem_ld16(to + C::TM_OX + q, ox);
                        tmem_ld16(to + C::TM_OI + q, oi);
                        uint4 wv[V / 8];
                        if constexpr (kRowAhead) {
                            // (rolled: the row's registers are picked by the turn)
#pragma unroll
                            for (int u = 0; u < V / 8; ++u)
                                wv[u] = q == 0 ? wrow[u] : q == 16 ? wrow[2 + u]
                                        : q == 32 ? wrow[4 + u] : wrow[6 + u];
                        } else if (kGrad && in && row_out) {
                            const uint4* src =
                                reinterpret_cast<const uint4*>(p.dot_with + grow * D + q);
#pragma unroll
                            for (int u = 0; u < V / 8; ++u) wv[u] = src[u];
                        }
                        tmem_ld_wait();
#pragma unroll
                        for (int u = 0; u < V; ++u) ox[u] = fmaf(rowf, ox[u], oi[u]);
                        if (__any_sync(0xffffffffu, !row_out)) {
#pragma unroll
                            for (int u = 0; u < V; ++u) ox[u] = row_out ? ox[u] : 0.f;
                        }
                        if (kGrad && in && row_out) {
#pragma unroll
                            for (int u = 0; u < V / 8; ++u) {
                                const uint32_t ww[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    dot = fmaf(ox[8 * u + 2 * r], __uint_as_float(ww[r] << 16), dot);
                                    dot = fmaf(ox[8 * u + 2 * r + 1],
                                               __uint_as_float(ww[r] & 0xffff0000u), dot);
                                }
                            }
                        }
                        const uint32_t base = tile + (q / 64) * C::kSub + row * 128;
#pragma unroll
                        for (int u = 0; u < V / 8; ++u) {
                            uint32_t pk[4];
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                pk[r] = pack_bf16(ox[8 * u + 2 * r], ox[8 * u + 2 * r + 1]);
                            st_shared16(base + ((((q % 64) / 8 + u) ^ (row & 7)) << 4), pk[0], pk[1],
                                        pk[2], pk[3]);
                        }
                    }
                    tc_fence_before();
                    cx.arrive(kOFree);
                    if (kGrad && in) p.dots[scratch_of(G, wk.it, wk.h, t)] = dot;
                    fence_proxy_async();
                    cx.arrive(kStore + at_.st);
                }
            }
            if (!ok) break;
            if (has_state) {
                if (kStateOnly) {
                    save_state(p.seg_state + seg_at);
                    if (sthread == 0)
                        p.seg_decay[(long long)wk.slot * G.H + wk.h] = ex2(logs);
                } else if (wk.ends) {
                    if (p.fin) save_state(p.fin + state_at);
                } else if (p.run > 0) {
                    float4* dst =
                        reinterpret_cast<float4*>(p.ho_state + (long long)blockIdx.x * D * D) + sthread;
#pragma unroll
                    for (int q = 0; q < R / 4; ++q)
                        __stcg(dst + q * kSThreads,
                               make_float4(S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]));
                    // each warp hands its own entries to the same warp of the next CTA
                    __threadfence();
                    __syncwarp();
                    if (lane == 0)
                        asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(
                                         p.ho_flag + 8 * (int)blockIdx.x + (sthread >> 5)),
                                     "r"(1u)
                                     : "memory");
                }
            }
        }
      };
      if (warp < 12)
          role(std::true_type{});
      else
          role(std::false_type{});
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// [B*T, H, D] bf16 as (D, H, B*T), box 64 x 1 x 128 rows; head first [B*H, T, D] as
// (D, T, B*H), box 64 x 128 x 1.  Either box lands as 128 swizzled rows of 128 bytes.
inline bool make_map(CUtensorMap* map, const void* ptr, int B, const Geom& g, int D) {
    chunked::EncodeTiledFn enc = chunked::encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)g.H, (cuuint64_t)B * g.T};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)g.H * D * 2};
    cuuint32_t box[3] = {64, 1, 128};
    if (g.head_first) {
        dims[1] = (cuuint64_t)g.T;
        dims[2] = (cuuint64_t)B * g.H;
        strides[1] = (cuuint64_t)g.T * D * 2;
        box[1] = 128;
        box[2] = 1;
    }
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device and the kernel's shared-memory size, set once per device.
template <int D, bool kRev, bool kStateOnly, bool kGrad>
inline int prepare_device() {
    constexpr int kMaxDev = 64;
    static std::atomic<int> sms[kMaxDev];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
    int n = sms[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
    if (cudaFuncSetAttribute(la_chunked_kernel<D, kRev, kStateOnly, kGrad>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<D>::kBytes) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    sms[dev].store(n, std::memory_order_release);
    return n;
}

template <int D, bool kRev, bool kStateOnly, bool kGrad>
inline cudaError_t launch_d(const Pass<__nv_bfloat16>& p, int B, cudaStream_t stream) {
    const int sms = prepare_device<D, kRev, kStateOnly, kGrad>();
    if (sms <= 0) {
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    }
    CUtensorMap m[4];
    const void* ptr[4] = {kStateOnly ? p.y : p.x, p.y, p.z, kStateOnly ? p.y : p.out};
    for (int i = 0; i < 4; ++i)
        if (!make_map(&m[i], ptr[i], B, p.geom, D)) return cudaErrorInvalidValue;
    const bool runs = !kStateOnly && p.run > 0;
    const long long items = p.geom.slots(runs ? kChunk : p.seg) * p.geom.H;
    const unsigned grid = (unsigned)(runs          ? (items + p.run - 1) / p.run
                                     : items < sms ? items
                                                   : sms);
    la_chunked_kernel<D, kRev, kStateOnly, kGrad><<<grid, kThreads, Cfg<D>::kBytes, stream>>>(m[0], m[1], m[2],
                                                                                 m[3], p);
    return cudaGetLastError();
}
template <bool kRev, bool kStateOnly>
inline cudaError_t launch_pass(const Pass<__nv_bfloat16>& p, int B, int D, cudaStream_t stream) {
    if constexpr (!kStateOnly) {
        if (p.dots)
            return D == 64 ? launch_d<64, kRev, false, true>(p, B, stream)
                           : launch_d<128, kRev, false, true>(p, B, stream);
    }
    return D == 64 ? launch_d<64, kRev, kStateOnly, false>(p, B, stream)
                   : launch_d<128, kRev, kStateOnly, false>(p, B, stream);
}

}  // namespace tc
}  // namespace la
}  // namespace wkv7
