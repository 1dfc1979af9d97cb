"""The operators around the biased attention, as measured cases: the gated
feed-forward block ("transition") of a pair, MSA or single representation, and
the learned relative-position bias that the attention takes as its pair bias,
each with its gradients.

    transition      Y = (act(X Wg^T) * (X Wu^T)) Wd^T
                    X, Y [M, C]; Wg, Wu [F, C]; Wd [C, F]; act: silu or gelu (erf)
    relative bias   P[b, 0, h, i, j] = table[r, h] (+ base[b, 0, h, i, j])
                    r = the number of borders <= pos_q[b, i] - pos_k[b, j], or the
                    table's last row where i and j lie in different chains

`run` computes a case in plain torch operations, or, where `own` is true, by the
package's entry points.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token's row of a single representation: all latency, 3.5 MB of weights to read
        dict(name="transition_token", op="transition", M=1, C=384, F=1536, act="silu", dtype="bf16"),
        # the single representation of an input of 1733 residues, channels that are no whole 16-byte units
        dict(name="transition_ragged", op="transition", M=1733, C=388, F=1555, act="silu", dtype="fp16"),
        # the MSA representation of 512 sequences x 256 residues (8 heads of 32)
        dict(name="transition_msa_512", op="transition", M=512 * 256, C=256, F=1024, act="silu", dtype="bf16"),
        # the pair representation of 768 residues, 128 channels: the size of the triangle multiplication's benchmark
        dict(name="transition_pair_768", op="transition", M=768 * 768, C=128, F=512, act="silu", dtype="bf16"),
        # a pair representation of 128 residues kept in fp32
        dict(name="transition_f32", op="transition", M=128 * 128, C=128, F=512, act="silu", dtype="fp32"),
        # training on the pair representation of 384 residues
        dict(name="transition_bwd_pair_384", op="transition_bwd", M=384 * 384, C=128, F=512, act="silu", dtype="bf16"),
        # training a wide block on 8192 tokens: compute-bound in every product
        dict(name="transition_bwd_wide", op="transition_bwd", M=8192, C=1024, F=4096, act="gelu", dtype="fp16"),
        # training with odd sizes everywhere
        dict(name="transition_bwd_ragged", op="transition_bwd", M=1009, C=100, F=397, act="gelu", dtype="bf16"),
        # the bias row of one new position against 1024 earlier ones, log-spaced buckets
        dict(name="relpos_row", op="relpos", B=1, Sq=1, Sk=1024, H=4, buckets="log", size=32, reach=128, chains=False, base=False, dtype="fp16"),
        # the bias of 2048 residues in several chains, added to a bias projected from the pair representation
        dict(name="relpos_2048", op="relpos", B=1, Sq=2048, Sk=2048, H=8, buckets="clip", size=32, reach=0, chains=True, base=True, dtype="bf16"),
        # the table's gradient from the pair-bias gradient of triangle attention at 1024 residues
        dict(name="relpos_bwd_1024", op="relpos_bwd", B=1, Sq=1024, Sk=1024, H=4, buckets="clip", size=32, reach=0, chains=True, base=False, dtype="bf16"),
        # the same in fp32 with 16 heads, log-spaced buckets and an odd length
        dict(name="relpos_bwd_1733", op="relpos_bwd", B=1, Sq=1733, Sk=1733, H=16, buckets="log", size=64, reach=512, chains=False, base=False, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["transition", "transition", "transition_bwd", "relpos", "relpos_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp16", "fp32"])
    if op.startswith("transition"):
        most = 128 * 128 * 128 * 512 if dtype == "fp32" else 768 * 768 * 128 * 512
        if op == "transition_bwd":  # 8 products of M x C x F for the forward's 3
            most = most * 3 // 8
        C = _log_int(rng, 16, 1024)
        if rng.random() < 0.6:
            C = max(16, C // 16 * 16)
        F = int(C * rng.choice([1.5, 2, 3.9, 4])) if rng.random() < 0.8 else _log_int(rng, 16, 4096)
        # neither more products nor more bytes than the largest listed case
        rows = 768 * 768 * 128 * 4 // (C * (4 if dtype == "fp32" else 2) * (3 if op == "transition_bwd" else 2))
        M = _log_int(rng, 1, max(1, min(768 * 768, rows, most // (C * F))))
        return dict(op=op, M=M, C=C, F=F, act=rng.choice(["silu", "silu", "gelu"]), dtype=dtype)
    B = rng.choice([1, 1, 1, 2, 3])
    H = rng.choice([1, 2, 3, 4, 8, 8, 16])
    Sq, Sk = _log_int(rng, 1, 2048), _log_int(rng, 1, 2048)
    if rng.random() < 0.6:
        Sq = Sk
    while B * H * Sq * Sk * (4 if dtype == "fp32" else 2) > 8 * 2048 * 2048 * 2:
        H, B = max(1, H // 2), max(1, B - 1)
    buckets = rng.choice(["clip", "log"])
    size = _log_int(rng, 1, 64) if buckets == "clip" else 2 * _log_int(rng, 4, 64)
    reach = 0 if buckets == "clip" else _log_int(rng, 2 * size, 40000)
    return dict(op=op, B=B, Sq=Sq, Sk=Sk, H=H, buckets=buckets, size=size, reach=reach, chains=rng.random() < 0.5,
                base=op == "relpos" and rng.random() < 0.5, dtype=dtype)


def _borders(case):
    """The sorted borders between the buckets of d = pos_q - pos_k, as integers."""
    if case["buckets"] == "clip":  # one bucket for each distance up to `size`, one more beyond it on each side
        return list(range(-case["size"], case["size"] + 1))
    # half of the `size` buckets for each sign: half of those for single distances, the
    # others for distances that grow by equal factors up to `reach`
    half = case["size"] // 2
    single, reach = half // 2, case["reach"]
    steps, up, t = half - single, [*range(1, single + 1)], single
    for k in range(1, steps):
        # the smallest t with (t / single)^steps >= (reach / single)^k, in whole numbers
        t = max(t, int(single * (reach / single) ** (k / steps)) - 2)
        while t ** steps * single ** k < reach ** k * single ** steps:
            t += 1
        up.append(t)
    up = sorted(set(up))
    return [1 - t for t in reversed(up)] + up


def _positions(rng, B, S, chains, start):
    """Residue numbers that run up with a gap here and there and begin anew in each
    chain, and the chains' numbers."""
    pos, chain = [], []
    for _ in range(B):
        ends = sorted(rng.randint(1, S) for _ in range(rng.randint(1, 4))) if chains else []
        p, c, at, cs = start, 0, [], []
        for i in range(S):
            if c < len(ends) and i == ends[c]:
                c, p = c + 1, rng.randint(0, 3)
                while c < len(ends) and i == ends[c]:
                    c += 1
            p += 1 if rng.random() > 0.02 else rng.randint(2, 20)
            at.append(p)
            cs.append(c)
        pos.append(at)
        chain.append(cs)
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return as_int(pos), as_int(chain) if chains else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]
    normal = lambda *shape, scale=1.0: (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)  # noqa: E731
    st = dict(case=dict(case))
    if case["op"].startswith("transition"):
        M, C, F = case["M"], case["C"], case["F"]
        st["x"] = normal(M, C)  # a layer norm comes before the block
        st["w_gate"], st["w_up"] = normal(F, C, scale=C ** -0.5), normal(F, C, scale=C ** -0.5)
        st["w_down"] = normal(C, F, scale=F ** -0.5)
        if case["op"] == "transition_bwd":
            st["dy"] = normal(M, C)
        return st
    B, Sq, Sk, H = case["B"], case["Sq"], case["Sk"], case["H"]
    rng = random.Random(seed * 1000003 + Sq * 31 + Sk)
    borders = _borders(case)
    st["borders"] = torch.tensor(borders, dtype=torch.int32, device="cuda")
    st["pos_k"], st["chain_k"] = _positions(rng, B, Sk, case["chains"], 0)
    if Sq == Sk:
        st["pos_q"], st["chain_q"] = st["pos_k"], st["chain_k"]
    else:  # the queries stand among the keys, or behind them
        st["pos_q"], st["chain_q"] = _positions(rng, B, Sq, case["chains"], rng.randint(0, Sk))
    rows = len(borders) + 1 + (1 if case["chains"] else 0)
    if case["op"] == "relpos":
        st["table"] = normal(rows, H)
        st["base"] = normal(B, 1, H, Sq, Sk) if case["base"] else None
    else:
        st["dpair"] = normal(B, 1, H, Sq, Sk)
        st["rows"] = rows
    return st


# ------------------------------------------------------------------ plain forms


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    phi = 0.5 * (1 + torch.erf(g * 2 ** -0.5))
    return g * phi, phi + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5


def _plain_transition(s):
    x, wg, wu, wd = (s[n].float() for n in ("x", "w_gate", "w_up", "w_down"))
    h = _act(x @ wg.T, s["case"]["act"])[0] * (x @ wu.T)
    return (h @ wd.T).to(s["x"].dtype)


def _plain_transition_bwd(s):
    x, wg, wu, wd, dy = (s[n].float() for n in ("x", "w_gate", "w_up", "w_down", "dy"))
    a, da = _act(x @ wg.T, s["case"]["act"])
    u, dh = x @ wu.T, dy @ wd
    dwd = dy.T @ (a * u)
    dg, du = dh * u * da, dh * a
    out = (dg @ wg + du @ wu, dg.T @ x, du.T @ x, dwd)
    return tuple(t.to(s["x"].dtype) for t in out)


def _plain_rows(s):
    """The table row of each pair, [B, Sq, Sk]."""
    d = s["pos_q"].long()[:, :, None] - s["pos_k"].long()[:, None, :]
    r = (d[..., None] >= s["borders"].long()).sum(-1)
    if s["chain_q"] is not None:
        r = torch.where(s["chain_q"][:, :, None] == s["chain_k"][:, None, :], r, s["borders"].numel() + 1)
    return r


def _plain_relpos(s):
    p = s["table"].float()[_plain_rows(s)].permute(0, 3, 1, 2)[:, None]
    return (p if s["base"] is None else p + s["base"].float()).to(s["table"].dtype).contiguous()


def _plain_relpos_bwd(s):
    H, R = s["case"]["H"], s["rows"]
    at = _plain_rows(s)[:, None] * H + torch.arange(H, device="cuda")[None, :, None, None]
    sums = torch.zeros(R * H, dtype=torch.float64, device="cuda")
    sums.index_add_(0, at.flatten(), s["dpair"].double().flatten())
    return sums.view(R, H).to(s["dpair"].dtype)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"transition": _plain_transition, "transition_bwd": _plain_transition_bwd, "relpos": _plain_relpos,
                "relpos_bwd": _plain_relpos_bwd}[c["op"]](s)
    import triangle_biased_attention_b200 as evo
    if c["op"] == "transition":
        return evo.transition(s["x"], s["w_gate"], s["w_up"], s["w_down"], act=c["act"])
    if c["op"] == "transition_bwd":
        return evo.transition_backward(s["x"], s["w_gate"], s["w_up"], s["w_down"], s["dy"], act=c["act"])
    if c["op"] == "relpos":
        return evo.relpos_bias(s["table"], s["borders"], s["pos_q"], s["pos_k"], s["chain_q"], s["chain_k"], base=s["base"])
    return evo.relpos_bias_backward(s["dpair"], s["borders"], s["pos_q"], s["pos_k"], s["chain_q"], s["chain_k"])


def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    if case["op"].startswith("transition"):
        M, C, F = case["M"], case["C"], case["F"]
        if case["op"] == "transition":  # x read, y written, three weights read
            return {"bytes": es * (2 * M * C + 3 * C * F), "flops": 6 * M * C * F}
        # x and dy read, dx written, three weights read and their gradients written
        return {"bytes": es * (3 * M * C + 6 * C * F), "flops": 16 * M * C * F}
    B, Sq, Sk, H = case["B"], case["Sq"], case["Sk"], case["H"]
    ids = (8 if case["chains"] else 4) * B * (Sq + Sk)
    nb = len(_borders(case))
    table = (nb + 1 + (1 if case["chains"] else 0)) * H * es
    pairs = B * H * Sq * Sk
    return {"bytes": pairs * es * (2 if case["base"] else 1) + table + ids + 4 * nb,
            "flops": pairs if case["base"] or case["op"] == "relpos_bwd" else 0}


# ------------------------------------------------------------- in 64 bits


def _exact_relpos_index(st):
    i = torch.searchsorted(st["borders"].long(), (st["pos_q"].long().unsqueeze(2) - st["pos_k"].long().unsqueeze(1)).contiguous(),
                           right=True)
    if st["chain_q"] is not None:
        i[st["chain_q"].unsqueeze(2) != st["chain_k"].unsqueeze(1)] = st["borders"].numel() + 1
    return i


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("transition"):
        wg, wu, wd = (st[n].double() for n in ("w_gate", "w_up", "w_down"))
        outs, sums = [], [torch.zeros_like(wg), torch.zeros_like(wu), torch.zeros_like(wd)]
        for r in range(0, case["M"], 65536):
            x = st["x"][r:r + 65536].double()
            gate, up = torch.einsum("mc,fc->mf", x, wg), torch.einsum("mc,fc->mf", x, wu)
            if case["act"] == "silu":
                sig = torch.sigmoid(gate)
                a, slope = gate * sig, sig + gate * sig * torch.sigmoid(-gate)
            else:
                cdf = 0.5 * torch.erfc(-gate / math.sqrt(2.0))
                a, slope = gate * cdf, cdf + gate * torch.exp(-gate.square() / 2) / math.sqrt(2 * math.pi)
            if case["op"] == "transition":
                outs.append(torch.einsum("mf,cf->mc", a * up, wd))
                continue
            dy = st["dy"][r:r + 65536].double()
            dh = torch.einsum("mc,cf->mf", dy, wd)
            dgate, dup = dh * up * slope, dh * a
            outs.append(torch.einsum("mf,fc->mc", dgate, wg) + torch.einsum("mf,fc->mc", dup, wu))
            sums[0] += torch.einsum("mf,mc->fc", dgate, x)
            sums[1] += torch.einsum("mf,mc->fc", dup, x)
            sums[2] += torch.einsum("mc,mf->cf", dy, a * up)
        y = torch.cat(outs)
        return y if case["op"] == "transition" else (y, *sums)
    i = _exact_relpos_index(st)
    if case["op"] == "relpos":
        p = torch.movedim(st["table"].double()[i], -1, 1).unsqueeze(1)
        return p if st["base"] is None else p + st["base"].double()
    v = st["dpair"].double().squeeze(1).movedim(1, -1).reshape(-1, case["H"])
    flat, order = torch.sort(i.flatten(), stable=True)
    # sums of each row's run, from differences of running sums of the rows in order
    run_ = torch.cat([torch.zeros_like(v[:1]), torch.cumsum(v[order], 0)])
    ends = torch.searchsorted(flat, torch.arange(st["rows"] + 1, device=flat.device))
    return run_[ends[1:]] - run_[ends[:-1]]
