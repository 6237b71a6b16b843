// la_api.inl -- the C ABI of the decay linear attention and layer norm entry points
// (include/wkv7.h): argument checks and dispatch.  Part of wkv7_api.cu.

namespace {

bool la_sizes_ok(int B, int T, int H, int K, int V, int N) {
    return B >= 0 && T >= 0 && H > 0 && K > 0 && V > 0 && N >= 0;
}
// Whether the tensor-core form exists.
bool la_chunked_ok(int K, wkv7_dtype dtype) { return dtype == WKV7_BF16 && K <= 128; }

// The problem behind the arguments, or a status.
wkv7_status la_problem(wkv7::la::Problem& p, int B, int T, int H, int K, int V, int packed,
                       const int32_t* cu, int N, int head_first, wkv7_dtype dtype,
                       wkv7_algo algo) {
    if (!la_sizes_ok(B, T, H, K, V, N)) return WKV7_ERR_INVALID_ARG;
    if (dtype != WKV7_BF16 && dtype != WKV7_F32) return WKV7_ERR_INVALID_ARG;
    if (algo != WKV7_ALGO_AUTO && algo != WKV7_ALGO_RECURRENT && algo != WKV7_ALGO_CHUNKED)
        return WKV7_ERR_INVALID_ARG;
    if (packed ? B != 1 : N != B) return WKV7_ERR_INVALID_ARG;
    if (!head_size_ok(K, V)) return WKV7_ERR_UNSUPPORTED;
    if (algo == WKV7_ALGO_CHUNKED && !la_chunked_ok(K, dtype)) return WKV7_ERR_UNSUPPORTED;
    // grids, TMA coordinates and slot numbers are 32-bit
    const long long units = (long long)N * H, tokens = (long long)B * T;
    if (tokens > 0x7ffffe00LL || units > 0x7fffffffLL / 16 ||
        (tokens / wkv7::la::kRecChunk + 2LL * N + 1) * H * (K / 64) > 0x7fffffffLL ||
        (long long)B * H > 0x7fffffffLL)
        return WKV7_ERR_UNSUPPORTED;
    p.geom = wkv7::la::Geom{cu, T, N, H, head_first};
    p.B = B;
    p.D = K;
    p.bf16 = dtype == WKV7_BF16;
    p.chunked = algo != WKV7_ALGO_RECURRENT && la_chunked_ok(K, dtype);
    return WKV7_OK;
}

// Test hook of the limits on the tensor-core kernel's waits (wkv7_test_hurry_next_la): taken by the
// next call that runs it.  Bit 31: set; bit 30: handoffs at once; the rest: nanoseconds.
std::atomic<unsigned> g_hurry{0};
void take_hurry(wkv7::la::Problem& p) {
    if (!p.chunked || p.geom.T == 0) return;
    const unsigned h = g_hurry.exchange(0);
    if (h == 0) return;
    p.wait_ns = h & 0x3fffffffu;
    p.handoff_at_once = (h >> 30) & 1;
}

// Workspace queries know whether the problem is packed, not where its offsets are: any
// non-null address makes the same plan.
const int32_t* la_some_cu(int packed) {
    return packed ? reinterpret_cast<const int32_t*>(uintptr_t{4}) : nullptr;
}

bool ok_workspace(const void* ws, size_t have, size_t need) {
    return need == 0 || (ok_ptr(ws) && have >= need);
}
wkv7_status status_of(cudaError_t e) { return e == cudaSuccess ? WKV7_OK : WKV7_ERR_CUDA; }

bool layout_ok(wkv7_layout l) { return l == WKV7_LAYOUT_BTHK || l == WKV7_LAYOUT_BHTK; }

// Whether p is one of the pointers.
template <typename... P>
bool one_of(const void* p, P... others) {
    return p && ((p == static_cast<const void*>(others)) || ...);
}

}  // namespace

extern "C" {

size_t wkv7_la_fwd_workspace_bytes(int B, int T, int H, int K, int V, int N, int packed,
                                   wkv7_dtype dtype, wkv7_algo algo) {
    wkv7::la::Problem p;
    if (la_problem(p, B, T, H, K, V, packed, la_some_cu(packed), N, 0, dtype, algo) != WKV7_OK)
        return 0;
    return wkv7::la::fwd_workspace(p);
}

wkv7_status wkv7_la_fwd(const void* q, const void* k, const void* v, const void* g, int g_per_head,
                        const float* s0, const uint8_t* mask, void* o, float* sT, int B, int T,
                        int H, int K, int V, const int32_t* cu_seqlens, int N, float scale,
                        wkv7_layout layout, wkv7_dtype dtype, wkv7_algo algo, void* workspace,
                        size_t workspace_bytes, void* stream_) {
    if (!layout_ok(layout) || !(scale - scale == 0.f)) return WKV7_ERR_INVALID_ARG;
    wkv7::la::Problem p;
    const wkv7_status st = la_problem(p, B, T, H, K, V, cu_seqlens != nullptr, cu_seqlens, N,
                                      layout == WKV7_LAYOUT_BHTK, dtype, algo);
    if (st != WKV7_OK) return st;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return WKV7_ERR_INVALID_ARG;
    const bool tokens = p.rows() > 0;
    if (tokens && (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) ||
                   !ok_scalar_ptr(g, dtype)))
        return WKV7_ERR_INVALID_ARG;
    if ((s0 && !aligned16(s0)) || (sT && !aligned16(sT))) return WKV7_ERR_INVALID_ARG;
    if (tokens && one_of(o, q, k, v, g)) return WKV7_ERR_INVALID_ARG;
    if (!ok_workspace(workspace, workspace_bytes, wkv7::la::fwd_workspace(p)))
        return WKV7_ERR_INVALID_ARG;
    if ((long long)N * H == 0) return WKV7_OK;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    take_hurry(p);
    auto run = [&](auto zero) {
        using T_ = decltype(zero);
        return wkv7::la::forward<T_>(p, static_cast<const T_*>(q), static_cast<const T_*>(k),
                                     static_cast<const T_*>(v), static_cast<const T_*>(g),
                                     g_per_head != 0, s0, mask, static_cast<T_*>(o), sT, scale,
                                     ws, stream);
    };
    return status_of(p.bf16 ? run(__nv_bfloat16()) : run(float()));
}

size_t wkv7_la_bwd_workspace_bytes(int B, int T, int H, int K, int V, int N, int packed,
                                   wkv7_dtype dtype, wkv7_algo algo) {
    wkv7::la::Problem p;
    if (la_problem(p, B, T, H, K, V, packed, la_some_cu(packed), N, 0, dtype, algo) != WKV7_OK)
        return 0;
    return wkv7::la::bwd_workspace(p);
}

wkv7_status wkv7_la_bwd(const void* q, const void* k, const void* v, const void* g, int g_per_head,
                        const float* s0, const uint8_t* mask, const void* dout, const float* dsT,
                        void* dq, void* dk, void* dv, void* dg, float* ds0, int B, int T, int H,
                        int K, int V, const int32_t* cu_seqlens, int N, float scale,
                        wkv7_layout layout, wkv7_dtype dtype, wkv7_algo algo, void* workspace,
                        size_t workspace_bytes, void* stream_) {
    if (!layout_ok(layout) || !(scale - scale == 0.f)) return WKV7_ERR_INVALID_ARG;
    wkv7::la::Problem p;
    const wkv7_status st = la_problem(p, B, T, H, K, V, cu_seqlens != nullptr, cu_seqlens, N,
                                      layout == WKV7_LAYOUT_BHTK, dtype, algo);
    if (st != WKV7_OK) return st;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return WKV7_ERR_INVALID_ARG;
    const bool tokens = p.rows() > 0;
    if (tokens && (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(dout) || !ok_ptr(dq) ||
                   !ok_ptr(dk) || !ok_ptr(dv) || !ok_scalar_ptr(g, dtype)))
        return WKV7_ERR_INVALID_ARG;
    if (dg && !ok_scalar_ptr(dg, dtype)) return WKV7_ERR_INVALID_ARG;
    if ((s0 && !aligned16(s0)) || (dsT && !aligned16(dsT)) || (ds0 && !aligned16(ds0)))
        return WKV7_ERR_INVALID_ARG;
    if (tokens && (one_of(dq, q, k, v, g, dout, dk, dv, dg) || one_of(dk, q, k, v, g, dout, dv, dg) ||
                   one_of(dv, q, k, v, g, dout, dg) || one_of(dg, q, k, v, g, dout)))
        return WKV7_ERR_INVALID_ARG;
    if (one_of(ds0, s0, dsT)) return WKV7_ERR_INVALID_ARG;
    if (!ok_workspace(workspace, workspace_bytes, wkv7::la::bwd_workspace(p)))
        return WKV7_ERR_INVALID_ARG;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if ((long long)N * H == 0) {  // no token: only the decays of the heads have a gradient, 0
        if (!dg || !g_per_head) return WKV7_OK;
        return status_of(cudaMemsetAsync(dg, 0, (size_t)H * (p.bf16 ? 2 : 4), stream));
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    take_hurry(p);
    auto run = [&](auto zero) {
        using T_ = decltype(zero);
        return wkv7::la::backward<T_>(
            p, static_cast<const T_*>(q), static_cast<const T_*>(k), static_cast<const T_*>(v),
            static_cast<const T_*>(g), g_per_head != 0, s0, mask, static_cast<const T_*>(dout),
            dsT, static_cast<T_*>(dq), static_cast<T_*>(dk), static_cast<T_*>(dv),
            static_cast<T_*>(dg), ds0, scale, ws, stream);
    };
    return status_of(p.bf16 ? run(__nv_bfloat16()) : run(float()));
}

wkv7_status wkv7_la_zero_tail(void* x0, void* x1, void* x2, void* scalars, int T, int H, int K,
                              const int32_t* cu_seqlens, int N, wkv7_layout layout,
                              wkv7_dtype dtype, void* stream_) {
    wkv7::la::Problem p;
    if (!layout_ok(layout)) return WKV7_ERR_INVALID_ARG;
    const wkv7_status st = la_problem(p, 1, T, H, K, K, 1, cu_seqlens, N,
                                      layout == WKV7_LAYOUT_BHTK, dtype, WKV7_ALGO_AUTO);
    if (st != WKV7_OK) return st;
    if (p.rows() == 0) return WKV7_OK;
    if (!cu_seqlens || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0 || !aligned16(x0) ||
        !aligned16(x1) || !aligned16(x2) || (scalars && !ok_scalar_ptr(scalars, dtype)))
        return WKV7_ERR_INVALID_ARG;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    auto run = [&](auto zero) {
        using T_ = decltype(zero);
        const wkv7::la::Tail<T_> t{{static_cast<T_*>(x0), static_cast<T_*>(x1), static_cast<T_*>(x2)},
                                   static_cast<T_*>(scalars), K};
        // 4 KB a block and turn; the tail's length is on the device
        const long long want = p.rows() * K / 2048 + 1;
        const unsigned blocks = (unsigned)(want < 296 ? want : 296);
        wkv7::la::la_tail_kernel<T_><<<blocks, 256, 0, stream>>>(p.geom, t);
        return cudaGetLastError();
    };
    return status_of(p.bf16 ? run(__nv_bfloat16()) : run(float()));
}

wkv7_status wkv7_la_step(const void* q, const void* k, const void* v, const void* g, int g_per_head,
                         const float* state, float* out_state, void* o, int B, int H, int K, int V,
                         float scale, wkv7_dtype dtype, void* stream_) {
    if (B < 0 || H <= 0 || K <= 0 || V <= 0 || !(scale - scale == 0.f)) return WKV7_ERR_INVALID_ARG;
    if (dtype != WKV7_BF16 && dtype != WKV7_F32) return WKV7_ERR_INVALID_ARG;
    if (!head_size_ok(K, V)) return WKV7_ERR_UNSUPPORTED;
    const long long units = (long long)B * H;
    if (units == 0) return WKV7_OK;
    if (units * (K / 64) > 0x7fffffffLL) return WKV7_ERR_UNSUPPORTED;
    if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(state) || !ok_ptr(out_state) ||
        !ok_ptr(o) || !ok_scalar_ptr(g, dtype))
        return WKV7_ERR_INVALID_ARG;
    if (one_of(o, q, k, v, g, state, out_state)) return WKV7_ERR_INVALID_ARG;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    return status_of(dtype == WKV7_BF16
                         ? wkv7::la::launch_la_step<__nv_bfloat16>(
                               q, k, v, g, g_per_head != 0, state, out_state, o, units, H, K,
                               scale, stream)
                         : wkv7::la::launch_la_step<float>(q, k, v, g, g_per_head != 0, state,
                                                           out_state, o, units, H, K, scale,
                                                           stream));
}

wkv7_status wkv7_test_hurry_next_la(int wait_ns, int handoff_at_once) {
    if (wait_ns < -1 || wait_ns > 1000000000) return WKV7_ERR_INVALID_ARG;
    g_hurry.store(wait_ns < 0 ? 0u
                              : 1u << 31 | (handoff_at_once ? 1u << 30 : 0u) | (unsigned)wait_ns);
    return WKV7_OK;
}

wkv7_status wkv7_test_la_pieces(int B, int T, int H, int K, const int32_t* cu_seqlens, int N,
                                wkv7_dtype dtype, int backward, int block, int32_t* pieces,
                                int max_pieces, int* count, int* blocks, int* skipped) {
    using namespace wkv7::la;
    if (!pieces || !count || !blocks || !skipped || max_pieces < 0 || block < 0)
        return WKV7_ERR_INVALID_ARG;
    Problem p;
    const wkv7_status st = la_problem(p, B, T, H, K, K, cu_seqlens != nullptr, cu_seqlens, N, 0,
                                      dtype, WKV7_ALGO_AUTO);
    if (st != WKV7_OK) return st;
    const Geom& g = p.geom;
    const Plan plan = make_plan(p);
    *count = *skipped = 0;
    for (int i = 0; cu_seqlens && i < N; ++i) *skipped |= seqlen_bad(g, i);
    // runs: a block each; segments (and all of the recurrent kernel's work): the whole list
    *blocks = plan.run > 0 ? (int)plan.blocks : 1;
    if (block >= *blocks) return WKV7_OK;
    tc::Cursor at = tc::first_cursor(g, plan.seg, plan.run, block);
    while (*count < max_pieces) {
        const tc::Piece s = tc::next_piece(g, plan.seg, at, backward != 0, 0);
        if (s.chunks < 0) break;
        const int32_t row[6] = {s.it.n, s.h, s.tb, s.te, s.begins, s.ends};
        for (int i = 0; i < 6; ++i) pieces[6 * *count + i] = row[i];
        ++*count;
    }
    return WKV7_OK;
}

// ---- layer norm -------------------------------------------------------------------------
// Whether p may hold rows (or weights of rows) of D elements of x's type: such rows are read and
// written in 16-byte groups where they are whole ones, and else by elements of `type`.
static bool ln_ptr(const void* p, int D, wkv7_dtype dtype, wkv7_dtype type) {
    const int group = dtype == WKV7_BF16 ? 8 : 4;
    return D % group == 0 ? ok_ptr(p) : ok_scalar_ptr(p, type);
}
static bool ln_stat_ptr(const float* p) { return !p || ok_scalar_ptr(p, WKV7_F32); }
static wkv7_status ln_check(long long rows, long long groups, long long inner, long long D,
                            wkv7_dtype dtype, wkv7_dtype wdtype) {
    if (rows < 0 || groups <= 0 || inner <= 0 || D <= 0) return WKV7_ERR_INVALID_ARG;
    if ((dtype != WKV7_BF16 && dtype != WKV7_F32) || (wdtype != WKV7_BF16 && wdtype != WKV7_F32))
        return WKV7_ERR_INVALID_ARG;
    if (dtype == WKV7_F32 && wdtype == WKV7_BF16) return WKV7_ERR_UNSUPPORTED;
    if (D > wkv7::ln::kMaxD || groups > 0x7fffffffLL || inner > 0x7fffffffLL ||
        groups > 0x7fffffffLL / D || rows > (1LL << 45) / D)
        return WKV7_ERR_UNSUPPORTED;
    // whole blocks of every group's rows
    if (rows % (groups * inner) != 0) return WKV7_ERR_INVALID_ARG;
    return WKV7_OK;
}

wkv7_status wkv7_ln_fwd(const void* x, const void* weight, const void* bias, void* y, float* mean,
                        float* rstd, int64_t rows, int groups, int64_t inner, int D, float eps,
                        wkv7_dtype dtype, wkv7_dtype wdtype, void* stream_) {
    const wkv7_status st = ln_check(rows, groups, inner, D, dtype, wdtype);
    if (st != WKV7_OK) return st;
    if (!(eps >= 0.f) || !(eps - eps == 0.f)) return WKV7_ERR_INVALID_ARG;
    if (rows == 0) return WKV7_OK;
    if (!ln_ptr(x, D, dtype, dtype) || !ln_ptr(y, D, dtype, dtype) ||
        (weight && !ln_ptr(weight, D, dtype, wdtype)) || (bias && !ln_ptr(bias, D, dtype, wdtype)) ||
        !ln_stat_ptr(mean) || !ln_stat_ptr(rstd))
        return WKV7_ERR_INVALID_ARG;
    if (one_of(y, x, weight, bias, mean, rstd) || one_of(mean, x, weight, bias, rstd) ||
        one_of(rstd, x, weight, bias))
        return WKV7_ERR_INVALID_ARG;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    auto run = [&](auto zx, auto zw) {
        using T_ = decltype(zx);
        using W_ = decltype(zw);
        return wkv7::ln::launch_fwd<T_, W_>(static_cast<const T_*>(x),
                                            static_cast<const W_*>(weight),
                                            static_cast<const W_*>(bias), static_cast<T_*>(y),
                                            mean, rstd, rows, groups, inner, D, eps, stream);
    };
    return status_of(dtype == WKV7_F32    ? run(float(), float())
                     : wdtype == WKV7_F32 ? run(__nv_bfloat16(), float())
                                          : run(__nv_bfloat16(), __nv_bfloat16()));
}

size_t wkv7_ln_bwd_workspace_bytes(int64_t rows, int groups, int64_t inner, int D,
                                   wkv7_dtype dtype) {
    if (ln_check(rows, groups, inner, D, dtype, WKV7_F32) != WKV7_OK || rows == 0) return 0;
    const long long S = dtype == WKV7_BF16 ? wkv7::ln::bwd_parts<__nv_bfloat16>(rows, groups, D)
                                           : wkv7::ln::bwd_parts<float>(rows, groups, D);
    return (size_t)S * 2 * groups * D * sizeof(float);
}

wkv7_status wkv7_ln_bwd(const void* x, const void* dy, const float* mean, const float* rstd,
                        const void* weight, void* dx, void* dweight, void* dbias, int64_t rows,
                        int groups, int64_t inner, int D, wkv7_dtype dtype, wkv7_dtype wdtype,
                        void* workspace, size_t workspace_bytes, void* stream_) {
    const wkv7_status st = ln_check(rows, groups, inner, D, dtype, wdtype);
    if (st != WKV7_OK) return st;
    if ((weight && !ln_ptr(weight, D, dtype, wdtype)) ||
        (dweight && !ln_ptr(dweight, D, dtype, wdtype)) ||
        (dbias && !ln_ptr(dbias, D, dtype, wdtype)))
        return WKV7_ERR_INVALID_ARG;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (rows == 0) {
        const size_t n = (size_t)groups * D * (wdtype == WKV7_BF16 ? 2 : 4);
        if (dweight && cudaMemsetAsync(dweight, 0, n, stream) != cudaSuccess) return WKV7_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, n, stream) != cudaSuccess) return WKV7_ERR_CUDA;
        return WKV7_OK;
    }
    if (!ln_ptr(x, D, dtype, dtype) || !ln_ptr(dy, D, dtype, dtype) || !ln_ptr(dx, D, dtype, dtype) ||
        !mean || !rstd || !ln_stat_ptr(mean) || !ln_stat_ptr(rstd))
        return WKV7_ERR_INVALID_ARG;
    if (one_of(dx, x, dy, weight, mean, rstd, dweight, dbias) || one_of(dweight, x, dy, weight, dbias) ||
        one_of(dbias, x, dy, weight))
        return WKV7_ERR_INVALID_ARG;
    if ((dweight || dbias) &&
        !ok_workspace(workspace, workspace_bytes,
                      wkv7_ln_bwd_workspace_bytes(rows, groups, inner, D, dtype)))
        return WKV7_ERR_INVALID_ARG;
    auto run = [&](auto zx, auto zw) {
        using T_ = decltype(zx);
        using W_ = decltype(zw);
        return wkv7::ln::launch_bwd<T_, W_>(
            static_cast<const T_*>(x), static_cast<const T_*>(dy), mean, rstd,
            static_cast<const W_*>(weight), static_cast<T_*>(dx), static_cast<W_*>(dweight),
            static_cast<W_*>(dbias), static_cast<float*>(workspace), rows, groups, inner, D,
            stream);
    };
    return status_of(dtype == WKV7_F32    ? run(float(), float())
                     : wdtype == WKV7_F32 ? run(__nv_bfloat16(), float())
                                          : run(__nv_bfloat16(), __nv_bfloat16()));
}

}  // extern "C"
