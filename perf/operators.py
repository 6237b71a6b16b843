"""The measured operators: linear attention with a decay for each head (whole sequences,
single tokens, gradients) and layer norm (over rows and per head, with its gradients).

Each case is one call of one operator.  ``run`` computes it either in its plain form
(elementary torch operations in 32 bits, the prefix sums of the log decays in 64) or, with
``own`` set, through this repository's public entry points.  ``exact`` is the same result
from the definition in 64 bits, token by token.

Linear attention, per (sequence, head), with a D x D state stored [k][v]:

    S_t = e^{g_t} S_{t-1} + k_t v_t^T        o_t = scale S_t^T q_t

and at a token whose mask is 0 the state stays and o_t = scale S_{t-1}^T q_t.  Layer norm of
a row x: y = (x - mean) rstd w + b, with one (w, b) for every row or one for each head.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CHUNK = 64


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # Training forward: the repository's headline shape (C = 4096 as 64 heads of 64),
        # a decay for each token and head, states in and out.
        dict(name="la_fwd_train_b8_t4096_h64", op="la_fwd", B=8, T=4096, H=64, D=64, seqs=0,
             dtype="bf16", gate="token", mask=False, s0=True, sT=True, hf=False),
        # One long prompt of a model with few, wide heads and a fixed decay for each head.
        dict(name="la_fwd_prompt_b1_t16384_h16_d128", op="la_fwd", B=1, T=16384, H=16, D=128,
             seqs=0, dtype="bf16", gate="head", mask=False, s0=False, sT=True, hf=False),
        # Prompts of many users packed into one row of tokens, some of them empty.
        dict(name="la_fwd_packed_64seq_h32", op="la_fwd", B=1, T=69565, H=32, D=64, seqs=64,
             dtype="bf16", gate="token", mask=False, s0=True, sT=True, hf=False),
        # A short fp32 call with an odd length and the head-first layout (latency counts).
        dict(name="la_fwd_fp32_b2_t333_h8_hf", op="la_fwd", B=2, T=333, H=8, D=64, seqs=0,
             dtype="fp32", gate="token", mask=True, s0=True, sT=True, hf=True),
        # Training backward at the headline shape.
        dict(name="la_bwd_train_b8_t4096_h64", op="la_bwd", B=8, T=4096, H=64, D=64, seqs=0,
             dtype="bf16", gate="token", mask=False, s0=True, sT=True, hf=False),
        # Fine-tuning a small batch of padded rows, wide heads, head-first, a fixed decay.
        dict(name="la_bwd_masked_b4_t1111_h16_d128_hf", op="la_bwd", B=4, T=1111, H=16, D=128,
             seqs=0, dtype="bf16", gate="head", mask=True, s0=False, sT=True, hf=True),
        # Decoding for 1024 users (the repository's decode shape).
        dict(name="la_step_b1024_h32", op="la_step", B=1024, H=32, D=64, dtype="bf16",
             gate="token"),
        # Decoding for one user: a latency case.
        dict(name="la_step_b1_h32_d128", op="la_step", B=1, H=32, D=128, dtype="bf16",
             gate="head"),
        # Layer norm in front of a mixing layer: rows of C = 4096.
        dict(name="ln_fwd_rows32768_d4096", op="ln_fwd", rows=32768, H=0, D=4096, dtype="bf16",
             wdtype="bf16", affine=True),
        # The per-head norm of a mixing layer's output, for a decode batch.
        dict(name="ln_fwd_heads_rows1024_h32_d64", op="ln_fwd", rows=1024, H=32, D=64,
             dtype="bf16", wdtype="fp32", affine=True),
        # Layer norm's backward over the same rows in training.
        dict(name="ln_bwd_rows32768_d4096", op="ln_bwd", rows=32768, H=0, D=4096, dtype="bf16",
             wdtype="fp32", affine=True),
        # An odd row length in fp32.
        dict(name="ln_bwd_fp32_rows3001_d1021", op="ln_bwd", rows=3001, H=0, D=1021,
             dtype="fp32", wdtype="fp32", affine=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_bwd", "la_step", "ln_fwd", "ln_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("la_fwd", "la_bwd"):
        D = rng.choice([64, 64, 128])
        packed = rng.random() < 0.3
        cap = 2 ** 25 if dtype == "bf16" else 2 ** 23
        while True:
            H = _log_int(rng, 4, 64)
            B = 1 if packed else _log_int(rng, 1, 16)
            T = _log_int(rng, 1, 20000)
            if B * T * H * D <= cap:
                break
        return dict(op=op, B=B, T=T, H=H, D=D, seqs=_log_int(rng, 1, 100) if packed else 0,
                    dtype=dtype, gate=rng.choice(["token", "head"]), mask=rng.random() < 0.4,
                    s0=rng.random() < 0.6, sT=rng.random() < 0.7,
                    hf=rng.random() < 0.3)
    if op == "la_step":
        D = rng.choice([64, 128, 256])
        H = _log_int(rng, 1, 64)
        B = _log_int(rng, 1, max(1, 2 ** 26 // (H * D * D)))
        return dict(op=op, B=B, H=H, D=D, dtype=dtype, gate=rng.choice(["token", "head"]))
    heads = rng.random() < 0.4
    H = _log_int(rng, 1, 64) if heads else 0
    D = rng.choice([64, 128, 256]) if heads else _log_int(rng, 1, 16384)
    rows = _log_int(rng, 1, max(1, min(60000, 2 ** 25 // (max(H, 1) * D))))
    return dict(op=op, rows=rows, H=H, D=D, dtype=dtype,
                wdtype="fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"]),
                affine=rng.random() < 0.85)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("la_fwd", "la_bwd"):
        N = case["seqs"] or case["B"]
        rows = case["B"] * case["T"] * case["H"]
        D = case["D"]
        state = N * case["H"] * D * D * 4
        tok = case["gate"] == "token"
        if op == "la_fwd":
            by = rows * (4 * D * es + (es if tok else 0))
            by += state * (int(case["s0"]) + int(case["sT"]))
            fl = 4 * D * D * rows
        else:
            by = rows * (7 * D * es + (2 * es if tok else 0))
            by += state * (2 * int(case["s0"]) + int(case["sT"]))
            fl = 10 * D * D * rows
        if case["mask"]:
            by += case["B"] * case["T"]
        return {"bytes": by, "flops": fl}
    if op == "la_step":
        u, D = case["B"] * case["H"], case["D"]
        return {"bytes": u * (8 * D * D + 4 * D * es + es), "flops": 5 * D * D * u}
    rows, D = case["rows"] * max(case["H"], 1), case["D"]
    wes = 2 if case["wdtype"] == "bf16" else 4
    nw = max(case["H"], 1) * D * int(case["affine"])
    if op == "ln_fwd":
        return {"bytes": 2 * rows * D * es + 8 * rows + 2 * nw * wes, "flops": 8 * rows * D}
    return {"bytes": 3 * rows * D * es + 8 * rows + 3 * nw * wes, "flops": 14 * rows * D}


# --------------------------------------------------------------------------------- inputs
def _cu_seqlens(T, n, rng):
    """n lengths that add up to T, spread over their logarithm; with 8 or more sequences one
    is empty."""
    w = [math.exp(rng.uniform(math.log(16.0), math.log(8192.0))) for _ in range(n)]
    if n >= 8:
        w[rng.randrange(n)] = 0.0
    total, acc, cu = sum(w), 0.0, [0]
    for x in w:
        acc += x
        cu.append(min(T, int(round(acc / total * T))))
    cu[-1] = T
    return cu


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    st = {"case": case}
    op = case["op"]
    if op in ("la_fwd", "la_bwd", "la_step"):
        H, D = case["H"], case["D"]
        if op == "la_step":
            lead, glead = (case["B"], H), (case["B"], H)
        elif case["hf"]:
            lead, glead = (case["B"], H, case["T"]), (case["B"], H, case["T"])
        else:
            lead, glead = (case["B"], case["T"], H), (case["B"], case["T"], H)
        st["q"] = randn(*lead, D).to(dt)
        k = randn(*lead, D)
        st["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
        del k
        st["v"] = randn(*lead, D).to(dt)
        if case["gate"] == "token":
            # log decays of the RWKV-7 range, (-0.607, 0)
            z = randn(*glead)
            st["g"] = (-torch.exp(-0.5 - torch.nn.functional.softplus(z))).to(dt)
        else:
            # a fixed decay for each head, memories of 32 tokens to some thousands
            e = 5.0 + 7.0 * torch.rand(H, device="cuda", generator=gen)
            st["g"] = torch.log1p(-torch.exp2(-e)).to(dt)
        st["scale"] = D ** -0.5
    if op == "la_step":
        st["state"] = 0.1 * randn(case["B"], H, D, D)
        st["out_state"] = torch.empty_like(st["state"])
        return st
    if op in ("la_fwd", "la_bwd"):
        B, T = case["B"], case["T"]
        rng = random.Random(seed)
        if case["seqs"]:
            cu = _cu_seqlens(T, case["seqs"], rng)
            st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            N = case["seqs"]
        else:
            cu, st["cu"], N = [T * i for i in range(B + 1)], None, B
        st["starts"], st["lens"] = cu[:-1], [b - a for a, b in zip(cu[:-1], cu[1:])]
        st["mask"] = None
        if case["mask"]:
            # a padded suffix for each row and 5% single tokens; of several rows one has
            # no live token at all
            m = torch.rand(B, T, device="cuda", generator=gen) >= 0.05
            pad = [rng.randrange(0, T // 4 + 1) for _ in range(B)]
            if B >= 3:
                pad[rng.randrange(B)] = T
            keep = torch.tensor([T - p for p in pad], device="cuda")[:, None]
            m &= torch.arange(T, device="cuda")[None] < keep
            st["mask"] = m.to(torch.uint8)
        st["s0"] = 0.1 * randn(N, H, D, D) if case["s0"] else None
        if op == "la_bwd":
            st["dout"] = randn(*lead, D).to(dt)
            st["dsT"] = 0.1 * randn(N, H, D, D) if case["sT"] else None
        return st
    shape = (case["rows"], case["H"], case["D"]) if case["H"] else (case["rows"], case["D"])
    wdt = _DT[case["wdtype"]]
    # activations of a residual stream: an offset and a spread of their own for each row
    lead = shape[:-1] + (1,)
    st["x"] = (randn(*shape) * torch.exp(0.5 * randn(*lead)) + 0.5 * randn(*lead)).to(dt)
    st["weight"] = st["bias"] = None
    if case["affine"]:
        st["weight"] = (1.0 + 0.2 * randn(*shape[1:])).to(wdt)
        st["bias"] = (0.2 * randn(*shape[1:])).to(wdt)
    st["eps"] = 1e-5
    if op == "ln_bwd":
        st["dy"] = randn(*shape).to(dt)
        # the statistics that the forward pass kept
        xf = st["x"].double()
        m = xf.mean(-1)
        st["mean"] = m.float()
        st["rstd"] = ((xf - m[..., None]).square().mean(-1) + st["eps"]).rsqrt().float()
    return st


# ----------------------------------------------------------------------- the plain forms
def _rows(x, hf):
    """[B,T,H,*] or [B,H,T,*] as [B T, H, *]."""
    if hf:
        x = x.transpose(1, 2)
    return x.reshape(x.shape[0] * x.shape[1], *x.shape[2:])


def _unrows(x, st):
    c = st["case"]
    x = x.reshape(c["B"], c["T"], *x.shape[1:])
    return x.transpose(1, 2).contiguous() if c["hf"] else x


class _Chunks:
    """The chunks of every sequence, one chunk of all sequences at a time."""

    def __init__(self, st):
        self.st = st
        self.hf = st["case"]["hf"]
        dev = st["q"].device
        self.start = torch.tensor(st["starts"], device=dev)[:, None]
        self.len = torch.tensor(st["lens"], device=dev)[:, None]
        self.n = -(-max(st["lens"], default=0) // _CHUNK)
        self.mask = None if st["mask"] is None else st["mask"].reshape(-1) != 0
        self.g = st["g"] if st["g"].dim() == 1 else _rows(st["g"], self.hf)

    def at(self, i):
        """Row numbers [N, C], which of them exist, which of them update the state, and the
        log decay's prefix sums [N, H, C] in 64 bits."""
        t = torch.arange(_CHUNK, device=self.start.device)[None] + i * _CHUNK
        ok = t < self.len
        idx = torch.where(ok, self.start + t, torch.zeros_like(t))
        live = ok if self.mask is None else ok & self.mask[idx]
        if self.g.dim() == 1:
            g = self.g.double()[None, :, None].expand(idx.shape[0], -1, idx.shape[1])
        else:
            g = self.g[idx].double().transpose(1, 2)
        return idx, ok, live, torch.where(live[:, None], g, torch.zeros_like(g)).cumsum(-1)

    @staticmethod
    def take(rows, idx, ok):
        x = rows[idx].float()                                   # [N, C, H, D]
        return torch.where(ok[..., None, None], x, torch.zeros_like(x)).transpose(1, 2)


def _decay(c, live):
    """e^{c_t - c_s} for s <= t where token s updates the state, else 0: [N, H, C, C]."""
    d = (c[..., :, None] - c[..., None, :])
    t = torch.arange(c.shape[-1], device=c.device)
    keep = (t[:, None] >= t[None]) & live[:, None, None, :]
    return torch.where(keep, torch.exp(d), torch.zeros_like(d)).float()


def _state0(st):
    c = st["case"]
    if st["s0"] is not None:
        return st["s0"]
    return torch.zeros(len(st["lens"]), c["H"], c["D"], c["D"], device=st["q"].device)


def _plain_la_fwd(st):
    ch = _Chunks(st)
    q, k, v = (_rows(st[n], ch.hf) for n in "qkv")
    out = torch.zeros(q.shape, dtype=torch.float32, device=q.device)
    S = _state0(st).clone()
    for i in range(ch.n):
        idx, ok, live, c = ch.at(i)
        qc, kc, vc = ch.take(q, idx, ok), ch.take(k, idx, live), ch.take(v, idx, live)
        ec = torch.exp(c).float()[..., None]
        o = (qc @ kc.transpose(-1, -2) * _decay(c, live)) @ vc + ec * (qc @ S)
        out[idx[ok]] = (st["scale"] * o).transpose(1, 2)[ok]
        tail = torch.exp(c[..., -1:] - c).float()[..., None]
        S = ec[..., -1:, :] * S + (tail * kc).transpose(-1, -2) @ vc
    return _unrows(out.to(st["q"].dtype), st), (S if st["case"]["sT"] else None)


def _plain_la_bwd(st):
    ch = _Chunks(st)
    q, k, v, do = (_rows(st[n], ch.hf) for n in ("q", "k", "v", "dout"))
    dq, dk, dv = (torch.zeros(q.shape, dtype=torch.float32, device=q.device) for _ in range(3))
    dg = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    scale = st["scale"]
    S = _state0(st)
    states = [S]
    for i in range(ch.n):
        idx, ok, live, c = ch.at(i)
        kc, vc = ch.take(k, idx, live), ch.take(v, idx, live)
        tail = torch.exp(c[..., -1:] - c).float()[..., None]
        S = torch.exp(c[..., -1:]).float()[..., None] * S + (tail * kc).transpose(-1, -2) @ vc
        states.append(S)
    G = torch.zeros_like(S) if st["dsT"] is None else st["dsT"]
    for i in range(ch.n - 1, -1, -1):
        idx, ok, live, c = ch.at(i)
        qc, kc, vc, dc = (ch.take(q, idx, ok), ch.take(k, idx, live), ch.take(v, idx, live),
                          ch.take(do, idx, ok))
        S1, S0 = states.pop(), states[-1]
        E = _decay(c, live)
        ec = torch.exp(c).float()[..., None]
        tail = torch.exp(c[..., -1:] - c).float()[..., None]
        P = qc @ kc.transpose(-1, -2) * E
        dP = dc @ vc.transpose(-1, -2) * E
        gq = scale * (dP @ kc + ec * (dc @ S0.transpose(-1, -2)))
        lv = live[:, None, :, None]
        gk = (scale * (dP.transpose(-1, -2) @ qc) + tail * (vc @ G.transpose(-1, -2))) * lv
        gv = (scale * (P.transpose(-1, -2) @ dc) + tail * (kc @ G)) * lv
        dc_t = (qc.double() * gq).sum(-1) - (kc.double() * gk).sum(-1)
        end = (S1.double() * G).sum((-1, -2))[..., None]
        gg = (dc_t.flip(-1).cumsum(-1).flip(-1) + end) * live[:, None]
        rows = idx[ok]
        dq[rows], dk[rows], dv[rows] = (x.transpose(1, 2)[ok] for x in (gq, gk, gv))
        dg[rows] = gg.transpose(1, 2)[ok]
        G = ec[..., -1:, :] * G + scale * (ec * qc).transpose(-1, -2) @ dc
    dt = st["q"].dtype
    dg = dg.sum(0) if st["g"].dim() == 1 else _unrows(dg, st)
    return (_unrows(dq.to(dt), st), _unrows(dk.to(dt), st), _unrows(dv.to(dt), st), dg.to(dt),
            G if st["case"]["s0"] else None)


def _plain_la_step(st):
    q, k, v = (st[n].float() for n in "qkv")
    d = torch.exp(st["g"].float())
    S = d[..., None, None] * st["state"] + k[..., :, None] * v[..., None, :]
    o = st["scale"] * (q[..., None, :] @ S)[..., 0, :]
    return o.to(st["q"].dtype), S


def _plain_ln_fwd(st):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + st["eps"])
    y = xc * rstd
    if st["weight"] is not None:
        y = y * st["weight"].float() + st["bias"].float()
    return y.to(st["x"].dtype), mean[..., 0], rstd[..., 0]


def _plain_ln_bwd(st):
    x, dy = st["x"].float(), st["dy"].float()
    xh = (x - st["mean"][..., None]) * st["rstd"][..., None]
    wdy = dy if st["weight"] is None else dy * st["weight"].float()
    dx = (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
    dx = (dx * st["rstd"][..., None]).to(st["x"].dtype)
    if st["weight"] is None:
        return dx, None, None
    wdt = st["weight"].dtype
    return dx, (dy * xh).sum(0).to(wdt), dy.sum(0).to(wdt)


_PLAIN = {"la_fwd": _plain_la_fwd, "la_bwd": _plain_la_bwd, "la_step": _plain_la_step,
          "ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd}


def run(st):
    """One call of the case's operator; returns its outputs."""
    case = st["case"]
    op = case["op"]
    if not own:
        return _PLAIN[op](st)
    import linear_attention_rnn_wkv7_b200 as lib
    if op == "la_fwd":
        return lib.wkv7_la_fwd(st["q"], st["k"], st["v"], st["g"], s0=st["s0"], mask=st["mask"],
                               cu_seqlens=st["cu"], output_final_state=case["sT"],
                               scale=st["scale"], head_first=case["hf"])
    if op == "la_bwd":
        r = lib.wkv7_la_bwd(st["q"], st["k"], st["v"], st["g"], st["dout"], s0=st["s0"],
                            mask=st["mask"], dsT=st["dsT"], cu_seqlens=st["cu"],
                            scale=st["scale"], head_first=case["hf"])
        return r["dq"], r["dk"], r["dv"], r["dg"], (r["ds0"] if case["s0"] else None)
    if op == "la_step":
        o = lib.wkv7_la_step(st["q"], st["k"], st["v"], st["g"], st["state"],
                             out_state=st["out_state"], scale=st["scale"])
        return o, st["out_state"]
    if op == "ln_fwd":
        return lib.wkv7_ln_fwd(st["x"], st["weight"], st["bias"], eps=st["eps"])
    r = lib.wkv7_ln_bwd(st["x"], st["dy"], st["mean"], st["rstd"], st["weight"])
    return r["dx"], r["dweight"], r["dbias"]


# ------------------------------------------------------------------ the definition, 64 bits
def _exact_tokens(st):
    """For step t of every sequence: rows [N], which sequences still run, which update."""
    dev = st["q"].device
    start, length = (torch.tensor(st[n], device=dev) for n in ("starts", "lens"))
    mask = None if st["mask"] is None else st["mask"].reshape(-1).bool()
    for t in range(max(st["lens"], default=0)):
        run_ = length > t
        row = torch.where(run_, start + t, torch.zeros_like(start))
        yield row, run_, (run_ if mask is None else run_ & mask[row])


def _exact_la(st, backward):
    hf = st["case"]["hf"]
    flat = {n: _rows(st[n], hf).double() for n in ("q", "k", "v", "dout") if n in st}
    alpha = torch.exp(st["g"].double())
    if alpha.dim() == 1:
        alpha = alpha[None].expand(flat["q"].shape[0], -1)
    else:
        alpha = _rows(alpha, hf)
    scale, case = st["scale"], st["case"]
    q, k, v = flat["q"], flat["k"], flat["v"]
    tokens = list(_exact_tokens(st))
    S = _state0(st).double()

    def advance(S, row, upd):
        new = alpha[row][..., None, None] * S + k[row][..., :, None] * v[row][..., None, :]
        return torch.where(upd[:, None, None, None], new, S)

    if not backward:
        out = torch.zeros_like(q)
        for row, run_, upd in tokens:
            S = advance(S, row, upd)
            o = scale * (q[row][..., None, :] @ S)[..., 0, :]
            out[row[run_]] = o[run_]
        return _unrows(out, st), (S if case["sT"] else None)

    do = flat["dout"]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    dg = torch.zeros_like(alpha, memory_format=torch.contiguous_format)
    span = 32                               # states kept every span tokens, rebuilt between
    kept = []
    for t, (row, run_, upd) in enumerate(tokens):
        if t % span == 0:
            kept.append(S)
        S = advance(S, row, upd)
    G = torch.zeros_like(S) if st["dsT"] is None else st["dsT"].double()
    for lo in range((len(kept) - 1) * span, -1, -span):
        part, before = tokens[lo:lo + span], [kept.pop()]
        for row, run_, upd in part:
            before.append(advance(before[-1], row, upd))
        for (row, run_, upd) in reversed(part):
            after = before.pop()
            live = run_[:, None, None, None]
            G = G + torch.where(live, scale * q[row][..., :, None] * do[row][..., None, :],
                                torch.zeros_like(G))
            gq = scale * (after @ do[row][..., None])[..., 0]
            gk = (G @ v[row][..., None])[..., 0]
            gv = (k[row][..., None, :] @ G)[..., 0, :]
            a = alpha[row]
            gg = a * (G * before[-1]).sum((-1, -2))
            dq[row[run_]] = gq[run_]
            dk[row[upd]], dv[row[upd]], dg[row[upd]] = gk[upd], gv[upd], gg[upd]
            G = torch.where(upd[:, None, None, None], a[..., None, None] * G, G)
    dg = dg.sum(0) if st["g"].dim() == 1 else _unrows(dg, st)
    return _unrows(dq, st), _unrows(dk, st), _unrows(dv, st), dg, (G if case["s0"] else None)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("la_fwd", "la_bwd"):
        steps, size = max(st["lens"], default=0), len(st["lens"]) * case["H"] * case["D"] ** 2
        # seconds: launches, and passes over the 64-bit states
        passes = 5 if op == "la_fwd" else 20
        if steps * passes * (2.5e-5 + 16.0 * size / 2.0e12) > 18.0:
            return None
        return _exact_la(st, op == "la_bwd")
    if op == "la_step":
        S = (torch.exp(st["g"].double())[..., None, None] * st["state"].double()
             + torch.einsum("bhk,bhv->bhkv", st["k"].double(), st["v"].double()))
        return st["scale"] * torch.einsum("bhkv,bhk->bhv", S, st["q"].double()), S
    x = st["x"].double()
    w = None if st["weight"] is None else st["weight"].double()
    if op == "ln_fwd":
        var, mean = torch.var_mean(x, dim=-1, correction=0)
        rstd = 1.0 / torch.sqrt(var + st["eps"])
        y = (x - mean.unsqueeze(-1)) * rstd.unsqueeze(-1)
        if w is not None:
            y = torch.addcmul(st["bias"].double(), y, w)
        return y, mean, rstd
    # the gradient of sum(y dy) for the statistics that the call is given
    dy, r = st["dy"].double(), st["rstd"].double().unsqueeze(-1)
    xh = (x - st["mean"].double().unsqueeze(-1)) * r
    u = dy if w is None else dy * w
    D = case["D"]
    dx = r / D * (D * u - u.sum(-1, keepdim=True) - xh * (u * xh).sum(-1, keepdim=True))
    if w is None:
        return dx, None, None
    return dx, torch.einsum("r...,r...->...", dy, xh), dy.sum(0)
