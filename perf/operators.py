"""What is measured of the serving path around MiniMax Sparse Attention: rotary positions, the paged
cache with its append, decode over the pages, and decode of a batch that shares a prefix.

Four kinds of cases, each one call of a public entry point:
  rope    rotates the query and key heads of T tokens (or, for training, takes the gradients back);
  append  rotates the new tokens' q, k, q_idx, k_idx and writes k, v, k_idx into the pages;
  decode  the 1..8 new tokens of every sequence select their blocks and attend, all from the pages;
  prefix  the same for sequences whose first tokens are one and the same run of pages.

The plain form computes them with elementary torch operations in 32 bits (angles in 64); index inputs are
small integers, as in the framework's workloads, so that scores and with them selections are exact.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def _rope(name, T, Hq, G, d, rot, dtype, interleaved, backward, stretch, far):
    return dict(name=name, kind="rope", T=T, Hq=Hq, G=G, d=d, rot=rot, dtype=dtype, interleaved=interleaved,
                backward=backward, stretch=stretch, far=far)


def _append(name, B, tokens, ragged, longest, Hq, G, d, d_idx, rot, ps, dtype, interleaved):
    return dict(name=name, kind="append", B=B, tokens=tokens, ragged=ragged, longest=longest, Hq=Hq, G=G, d=d,
                d_idx=d_idx, rot=rot, ps=ps, dtype=dtype, interleaved=interleaved)


def _decode(name, B, S, longest, ragged, padded, Hq, G, d, d_idx, k, bk, ps, prefix=0):
    return dict(name=name, kind="prefix" if prefix else "decode", B=B, S=S, longest=longest, ragged=ragged,
                padded=padded, Hq=Hq, G=G, d=d, d_idx=d_idx, k=k, bk=bk, ps=ps, prefix=prefix)


def listed():
    return [
        # one decode step of 64 sequences at the workload's heads: latency, positions far out, YaRN
        _rope("rope-step-64", 64, 64, 8, 128, 128, "bf16", False, False, "yarn", 131072),
        # the prompt of the 32K workload
        _rope("rope-prompt-32k", 32768, 64, 8, 128, 128, "bf16", False, False, "ntk", 32768),
        # a training step's gradients in fp32: odd length, interleaved pairs, half of each head rotated
        _rope("rope-grad-4097-fp32", 4097, 8, 2, 64, 32, "fp32", True, True, "linear", 4097),
        # the new tokens of one decode step, short caches of the tiny configuration
        _append("append-step-8-tiny", 8, 1, False, 300, 8, 2, 64, 32, 32, 16, "bf16", True),
        # the same at the workload's heads, 64 sequences
        _append("append-step-64", 64, 1, False, 500, 64, 8, 128, 128, 64, 64, "bf16", False),
        # a chunk of a few prompts of different lengths
        _append("append-chunk-8191", 5, 8191, True, 4000, 64, 8, 128, 128, 128, 16, "bf16", False),
        # one short sequence: latency
        _decode("decode-1-700-tiny", 1, 1, 700, False, 0, 8, 2, 64, 32, 4, 128, 16),
        # a serving batch of mixed lengths with padded rows
        _decode("decode-32-16k-ragged", 32, 1, 16384, True, 3, 64, 8, 128, 128, 16, 128, 64),
        # few sequences, the cache of the 128K workload
        _decode("decode-8-128k", 8, 1, 131073, False, 0, 64, 8, 128, 128, 16, 128, 128),
        # a short system prompt shared by a few requests; blocks of 32
        _decode("prefix-6-1k-bk32", 6, 1, 1500, True, 0, 16, 4, 128, 64, 8, 32, 16, 1008),
        # four drafted tokens a sequence behind a shared document
        _decode("prefix-16x4-32k", 16, 4, 34000, True, 1, 64, 8, 128, 128, 16, 128, 64, 32768),
        # the workload's decode batch, all behind one 128K document
        _decode("prefix-64-128k", 64, 1, 133000, True, 0, 64, 8, 128, 128, 16, 128, 64, 131072),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# (Hq, G, d, d_idx): the framework's two configurations and shapes between them
HEADS = ((8, 2, 64, 32), (16, 4, 128, 64), (64, 8, 128, 128), (16, 1, 128, 128), (8, 8, 64, 64), (12, 3, 128, 32))


def draw(rng):
    kind = rng.choice(("rope", "append", "decode", "prefix"))
    Hq, G, d, d_idx = rng.choice(HEADS)
    ps = rng.choice((16, 32, 64, 128))
    if kind == "rope":
        rot = rng.choice((d, d, d // 2, d // 4, d // 2 + 4, d - 10))
        c = _rope("", _log(rng, 1, 20000), Hq, G, d, rot, rng.choice(("bf16", "fp16", "fp32")), rng.random() < 0.5,
                  rng.random() < 0.4, rng.choice(("none", "linear", "ntk", "yarn")), _log(rng, 1000, 1 << 20))
    elif kind == "append":
        B = _log(rng, 1, 200)
        ragged = rng.random() < 0.5
        tokens = _log(rng, B, 8000) if ragged else rng.choice((1, 1, 2, 5))
        c = _append("", B, tokens, ragged, _log(rng, 64, 400000 // B // 4), Hq, G, d, d_idx,
                    rng.choice((d_idx, d_idx // 2, 20)), ps, rng.choice(("bf16", "bf16", "fp16", "fp32")),
                    rng.random() < 0.5)
    else:
        S = rng.choice((1, 1, 2, 4, 8))
        B = _log(rng, 1, 64 // S)
        bk, k = rng.choice((32, 64, 128)), rng.choice((1, 4, 8, 13, 16, 32))
        if kind == "decode":
            c = _decode("", B, S, _log(rng, 40, 500000 // B), rng.random() < 0.7, rng.choice((0, 0, 1)) if B > 1 else 0,
                        Hq, G, d, d_idx, k, bk, ps)
        else:
            prefix = ps * max(1, _log(rng, 200, 100000) // ps)
            c = _decode("", B, S, prefix + _log(rng, 20, 20000 // B + 40), rng.random() < 0.7,
                        rng.choice((0, 0, 1)) if B > 1 else 0, Hq, G, d, d_idx, k, bk, ps, prefix)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs
def _frequencies(rot, stretch):
    """(radians a position for every pair, what cos and sin are multiplied with)."""
    base, factor, trained = 10000.0, 8.0, 4096
    if stretch == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    scale = 1.0
    if stretch == "linear":
        f = [x / factor for x in f]
    if stretch == "yarn":   # pairs that turn over 32 times in the trained length keep their frequency, under once are stretched
        turns = [trained * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (math.log(t) - 0.0) / math.log(32.0))) for t in turns]
        f = [x * (w + (1 - w) / factor) for x, w in zip(f, keep)]
        scale = 0.1 * math.log(factor) + 1.0
    return f, scale


def _fresh(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if math.prod(shape) < 1 << 26 else dtype).to(dtype)


def _whole(gen, shape, a):
    """Integers in [-a, a] as bf16: index inputs whose dot products are exact."""
    return torch.randint(-a, a + 1, shape, generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)


def _lengths(case, gen, least):
    B, longest = case["B"], case["longest"]
    n = torch.full((B,), longest, dtype=torch.int64, device="cuda")
    if case["ragged"] and B > 1:
        n = least + torch.randint(0, longest - least + 1, (B,), generator=gen, device="cuda")
        n[0] = longest
    return n


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["kind"] == "rope":
        dtype = TYPES[case["dtype"]]
        f, s["scale"] = _frequencies(case["rot"], case["stretch"])
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        T = case["T"]
        # a prompt or training sequence: consecutive; a decode step: each token somewhere else
        s["positions"] = (torch.randint(0, case["far"], (T,), generator=gen, device="cuda") if T <= 256 else
                          torch.randint(0, max(1, case["far"] - T) + 1, (1,), generator=gen, device="cuda") + torch.arange(T, device="cuda"))
        # the heads as slices of one projection's output, as a model has them
        qk = _fresh(gen, (T, (case["Hq"] + case["G"]) * case["d"]), dtype)
        s["q"] = qk[:, :case["Hq"] * case["d"]].unflatten(1, (case["Hq"], case["d"]))
        s["k"] = qk[:, case["Hq"] * case["d"]:].unflatten(1, (case["G"], case["d"]))
        s["out"] = tuple(torch.empty(x.shape, dtype=dtype, device="cuda") for x in (s["q"], s["k"]))
        return s
    B, ps, Hq, G, d, di = (case[x] for x in ("B", "ps", "Hq", "G", "d", "d_idx"))
    bf16 = torch.bfloat16
    if case["kind"] == "append":
        dtype = TYPES[case["dtype"]]
        if case["ragged"]:   # a chunk of the whole is cut at random places; some sequences may get nothing
            total = case["tokens"]
            cuts = torch.randint(0, total + 1, (B - 1,), generator=gen, device="cuda").sort().values
            s["cu_seqlens"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), total)]).to(torch.int32)
            new = s["cu_seqlens"].diff().long()
            T, capacity = total, case["longest"] + total
        else:
            new = torch.full((B,), case["tokens"], dtype=torch.int64, device="cuda")
            s["cu_seqlens"] = None
            T, capacity = B * case["tokens"], case["longest"] + case["tokens"]
        before = torch.randint(0, case["longest"] + 1, (B,), generator=gen, device="cuda")
        s["seqlens"] = (before + new).to(torch.int32)
        # the pages that each sequence needs, as a pool deals them out
        pages = -(-(before + new) // ps)
        most = -(-capacity // ps)
        room = (B * case["longest"] + T) // ps + B
        order = torch.randperm(room + 3, generator=gen, device="cuda").to(torch.int32)
        first = pages.cumsum(0) - pages
        at = first[:, None] + torch.arange(most, device="cuda")
        held = torch.arange(most, device="cuda") < pages[:, None]
        s["page_table"] = torch.where(held, order[at.clamp(max=room - 1)], -1).contiguous()
        for name, w in (("k_pages", d), ("v_pages", d), ("k_idx_pages", di)):
            s[name] = torch.zeros(room + 3, ps, G, w, dtype=bf16, device="cuda")
        for name, h, w in (("q", Hq, d), ("k", G, d), ("v", G, d), ("q_idx", G, di), ("k_idx", G, di)):
            s[name] = _fresh(gen, (T, h, w), dtype)
        f, s["scale"] = _frequencies(case["rot"], "yarn")
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["out"] = (torch.zeros(T, Hq, d, dtype=bf16, device="cuda"), torch.zeros(T, G, di, dtype=bf16, device="cuda"))
    else:
        S, prefix = case["S"], case["prefix"]
        n = _lengths(case, gen, max(S, prefix + S if prefix else case["longest"] // 4))
        n[B - case["padded"]:] = 0   # rows of a batch that is padded to its captured size
        s["seqlens"] = n.to(torch.int32)
        most, shared = -(-case["longest"] // ps), prefix // ps
        room = B * (most - shared) + shared
        order = torch.randperm(room + 1, generator=gen, device="cuda").to(torch.int32)
        s["prefix_pages"] = order[:shared].contiguous() if prefix else None
        own_pages = order[shared:room].view(B, most - shared)
        s["page_table"] = torch.cat([order[:shared].expand(B, shared), own_pages], 1).contiguous()
        s["k_pages"], s["v_pages"] = (_fresh(gen, (room + 1, ps, G, d), bf16) for _ in range(2))
        ki = _whole(gen, (room + 1, ps, G, di), 4)
        hot = torch.rand(room + 1, 1, 1, 1, generator=gen, device="cuda") < 0.05   # pages that many queries look for
        s["k_idx_pages"] = ki.add_(torch.where(hot, _whole(gen, (1, 1, G, di), 2), 0.0))
        s["q"] = _fresh(gen, (B, S, Hq, d), bf16)
        s["q_idx"] = _whole(gen, (B, S, G, di), 4)
        s["out"] = (torch.empty_like(s["q"]), torch.empty(B, S, G, case["k"], dtype=torch.int32, device="cuda"))
    if own:   # the handle that a serving program makes once for its cache, and its workspace
        from block_sparse_long_tcgen05_b200 import msa
        s["cache"] = msa.PagedCache(s["k_pages"], s["v_pages"], s["k_idx_pages"])
        if case["kind"] != "append":
            need = msa.paged_decode_workspace(s["cache"], B, s["page_table"].shape[1], Hq, case["k"], bk=case["bk"],
                                              n_new=case["S"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    kind = s["kind"]
    if own:
        from block_sparse_long_tcgen05_b200 import msa
        if kind == "rope":
            return msa.rope((s["q"], s["k"]), s["positions"], s["freqs"], interleaved=s["interleaved"],
                            scale=s["scale"], backward=s["backward"], out=s["out"])
        if kind == "append":
            msa.paged_append(s["cache"], s["page_table"], s["seqlens"], s["k"], s["v"], s["k_idx"],
                             cu_seqlens=s["cu_seqlens"], freqs=s["freqs"], interleaved=s["interleaved"],
                             rope_scale=s["scale"], q=s["q"], q_idx=s["q_idx"], q_out=s["out"][0], q_idx_out=s["out"][1])
            return s["out"] + (s["k_pages"], s["v_pages"], s["k_idx_pages"])
        msa.paged_decode(s["cache"], s["page_table"], s["seqlens"], s["q"], s["q_idx"], s["k"], bk=s["bk"],
                         prefix_pages=s["prefix_pages"], block_ids=s["out"][1], o=s["out"][0], workspace=s["workspace"])
        return s["out"]
    if kind == "rope":
        return tuple(_rotate(s[x], s["positions"], s["freqs"], s["interleaved"], s["scale"], s["backward"]) for x in ("q", "k"))
    if kind == "append":
        return _plain_append(s)
    return _plain_decode(s)


def _rotate(x, positions, freqs, interleaved, scale, backward=False, dtype=None):
    """The first 2 * len(freqs) elements of every head rotated, the rest as they are."""
    rot, h = 2 * freqs.numel(), freqs.numel()
    angle = positions.double()[:, None, None] * freqs
    c, n = (angle.cos() * scale).float(), (angle.sin() * (-scale if backward else scale)).float()
    y = x.float()
    head = y[..., :rot]
    a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else (head[..., :h], head[..., h:])
    ya, yb = a * c - b * n, a * n + b * c
    turned = torch.stack((ya, yb), -1).flatten(-2) if interleaved else torch.cat((ya, yb), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(dtype or x.dtype)


def _plain_append(s):
    B, ps = s["B"], s["ps"]
    T = s["k"].shape[0]
    t = torch.arange(T, device="cuda")
    if s["cu_seqlens"] is None:
        new = T // B
        seq, end = t // new, (t // new + 1) * new
    else:
        cu = s["cu_seqlens"].long()
        seq = torch.searchsorted(cu[1:], t, right=True)
        end = cu[seq + 1]
    pos = s["seqlens"].long()[seq] - (end - t)
    slot = s["page_table"].long()[seq, pos // ps] * ps + pos % ps
    turn = lambda x: _rotate(x, pos, s["freqs"], s["interleaved"], s["scale"], dtype=torch.bfloat16)  # noqa: E731
    s["k_pages"].flatten(0, 1)[slot] = turn(s["k"])
    s["v_pages"].flatten(0, 1)[slot] = s["v"].to(torch.bfloat16)
    s["k_idx_pages"].flatten(0, 1)[slot] = turn(s["k_idx"])
    return turn(s["q"]), turn(s["q_idx"]), s["k_pages"], s["v_pages"], s["k_idx_pages"]


def _plain_decode(s):
    B, S, Hq, G, d, di, k, bk, ps, prefix = (s[x] for x in ("B", "S", "Hq", "G", "d", "d_idx", "k", "bk", "ps", "prefix"))
    table = s["page_table"].long()
    shared = prefix // ps
    pos = s["seqlens"].long()[:, None] - S + torch.arange(S, device="cuda")          # [B, S], negative: no token
    L = table.shape[1] * ps
    nb = -(-L // bk)
    # token scores: the shared pages once for all rows, each sequence's own pages for its rows
    qi = s["q_idx"].float()
    keys = s["k_idx_pages"][table[:, shared:]].float().flatten(1, 2)                 # [B, own tokens, G, di]
    score = torch.matmul(qi.transpose(1, 2), keys.permute(0, 2, 3, 1))               # [B, G, S, own tokens]
    if shared:
        first = s["k_idx_pages"][s["prefix_pages"].long()].float().flatten(0, 1)     # [prefix tokens, G, di]
        every = torch.matmul(qi.permute(2, 0, 1, 3).flatten(1, 2), first.permute(1, 2, 0))   # [G, B * S, prefix tokens]
        score = torch.cat((every.unflatten(1, (B, S)).transpose(0, 1), score), -1)
    score = score.transpose(1, 2)                                                    # [B, S, G, L]
    seen = (torch.arange(L, device="cuda") <= pos[..., None])[:, :, None]
    score = torch.nn.functional.pad(score.masked_fill(~seen, -math.inf), (0, nb * bk - L), value=-math.inf)
    best = score.unflatten(-1, (nb, bk)).amax(-1)                                    # [B, S, G, nb]
    # the local block and the k - 1 best others; equal scores: the lower block first
    local = torch.div(pos, bk, rounding_mode="floor")[..., None, None]
    block = torch.arange(nb, device="cuda")
    best = torch.where(block == local, math.inf, best)
    ids = best.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    if nb < k:
        ids = torch.cat((ids, ids.new_full((B, S, G, k - nb), nb)), -1)
    ids = torch.where(ids > local, nb, ids).sort(-1).values
    taken = ids < nb
    # attention over the tokens of the chosen blocks
    token = (ids[..., None] * bk + torch.arange(bk, device="cuda")).flatten(-2)      # [B, S, G, k * bk]
    real = taken.repeat_interleave(bk, -1) & (token <= pos[..., None, None])
    token = torch.where(real, token, 0)
    page = table[torch.arange(B, device="cuda")[:, None, None, None], token // ps]
    slot = page * ps + token % ps
    group = torch.arange(G, device="cuda")[:, None]
    kk = s["k_pages"].flatten(0, 1)[slot, group].float()                             # [B, S, G, k * bk, d]
    vv = s["v_pages"].flatten(0, 1)[slot, group].float()
    logit = torch.matmul(s["q"].float().unflatten(2, (G, Hq // G)), kk.transpose(-1, -2)) / math.sqrt(d)
    logit = logit.masked_fill(~real[..., None, :], -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(top == -math.inf, 0.0, top))
    o = torch.matmul(p, vv) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.flatten(2, 3).to(torch.bfloat16), torch.where(taken, ids, -1).to(torch.int32)


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and row by row."""
    s = prepare(case, seed)
    if case["kind"] == "rope":
        return [_turned(s[x].double(), s["positions"], s) for x in ("q", "k")]
    table, ps = s["page_table"].tolist(), case["ps"]
    lengths = s["seqlens"].tolist()
    if case["kind"] == "append":
        T = s["k"].shape[0]
        cu = s["cu_seqlens"].tolist() if case["ragged"] else [b * case["tokens"] for b in range(case["B"] + 1)]
        pos, slot = [0] * T, [0] * T
        for b in range(case["B"]):
            for t in range(cu[b], cu[b + 1]):
                pos[t] = lengths[b] - cu[b + 1] + t
                slot[t] = table[b][pos[t] // ps] * ps + pos[t] % ps
        at, where = torch.tensor(pos, device="cuda"), torch.tensor(slot, device="cuda")
        pools = []
        for name, turned in (("k", True), ("v", False), ("k_idx", True)):
            pool = s[name + "_pages"].double()
            x = s[name].double()
            pool.view(-1, *x.shape[1:]).index_copy_(0, where, _turned(x, at, s) if turned else x)
            pools.append(pool)
        return [_turned(s["q"].double(), at, s), _turned(s["q_idx"].double(), at, s)] + pools
    B, S, G, k, bk, R = case["B"], case["S"], case["G"], case["k"], case["bk"], case["Hq"] // case["G"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    ids = torch.full((B, S, G, k), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        n = lengths[b]
        if n == 0:
            continue
        pages = torch.tensor(table[b][:-(-n // ps)], device="cuda")
        ki, kc, vc = (s[x][pages].view(-1, G, s[x].shape[-1])[:n] for x in ("k_idx_pages", "k_pages", "v_pages"))
        for r in range(S):
            at = n - S + r
            if at < 0:
                continue
            lb = at // bk
            for g in range(G):
                if lb + 1 <= k:
                    chosen = list(range(lb + 1))
                else:
                    best = (ki[:lb * bk, g].double() @ s["q_idx"][b, r, g].double()).view(lb, bk).max(1).values
                    # one key for score and block: whole scores, the lower block first
                    key = best * (1 << 32) - torch.arange(lb, dtype=torch.float64, device="cuda")
                    chosen = sorted(torch.topk(key, k - 1).indices.tolist() + [lb])
                ids[b, r, g, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
                token = torch.tensor(chosen, device="cuda")[:, None] * bk + torch.arange(bk, device="cuda")
                token = token.flatten()
                token = token[token <= at]
                w = torch.softmax(s["q"][b, r, g * R:(g + 1) * R].double() @ kc[token, g].double().T / math.sqrt(case["d"]), -1)
                o[b, r, g * R:(g + 1) * R] = w @ vc[token, g].double()
    return [o, ids]


def _turned(x, positions, s):
    """Each pair as a complex number times scale * exp(+-i * position * frequency)."""
    f = s["freqs"]
    w = torch.polar(torch.full_like(f, s["scale"]).expand(len(positions), -1).contiguous(), positions.double()[:, None] * f)[:, None]
    w = w.conj() if s.get("backward") else w
    m = 2 * len(f)
    pairs = x[..., :m].unflatten(-1, (-1, 2)) if s["interleaved"] else x[..., :m].unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    return torch.cat(((z if s["interleaved"] else z.transpose(-1, -2)).flatten(-2), x[..., m:]), -1)


# ------------------------------------------------------------------------------------ work
def work(case):
    e = 4 if case.get("dtype") == "fp32" else 2
    if case["kind"] == "rope":
        n = case["T"] * (case["Hq"] + case["G"])
        return {"bytes": 2 * n * case["d"] * e + 8 * case["T"], "flops": 3 * n * case["rot"]}
    Hq, G, d, di, B, ps = (case[x] for x in ("Hq", "G", "d", "d_idx", "B", "ps"))
    if case["kind"] == "append":
        T = case["tokens"] if case["ragged"] else B * case["tokens"]
        return {"bytes": T * (Hq * d + 2 * G * d + 2 * G * di) * (e + 2), "flops": 3 * T * (Hq + 3 * G) * case["rot"]}
    # index keys before the local block: a shared prefix once, each sequence's own part; the chosen blocks, at most all there are
    S, k, bk, prefix = case["S"], case["k"], case["bk"], case["prefix"]
    live = B - case["padded"]
    least = max(S, prefix + S if prefix else case["longest"] // 4)
    mean = (case["longest"] + least) / 2 if case["ragged"] and B > 1 else case["longest"]
    own_tokens = live * (mean - prefix)
    chosen = live * S * min(k * bk, mean)
    kv = min(chosen, prefix + own_tokens) * G * 4 * d
    io = live * S * (2 * Hq * d + G * di) * 2 + live * S * G * k * 4
    flops = 2 * G * di * live * S * mean + 4 * Hq * d * chosen
    return {"bytes": (prefix + own_tokens) * G * di * 2 + kv + io, "flops": flops}
