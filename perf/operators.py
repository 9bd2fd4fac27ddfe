"""What the linear-attention and page operators are measured on.

Linear attention with a decay for each head, over packed sequences (token-major, offsets in
``cu_seqlens``), S_t = exp(g_t) S_{t-1} + k_t v_t^T and o_t = scale S_t^T q_t per head: the forward
over prompts, its backward, and the step of one token on states that live in the pages of a pool;
and the operators on such a pool's pages: fork, compact, free.

``run`` computes them from elementary torch operations in 32 bits (``own`` false) or by the
library's calls (``own`` true).  Sizes follow the packed, long, fork and training workloads of
``gdn_inputs.py`` and the benchmark's decode step.
"""
import random

import torch

own = False

CHUNK = 64  # block length of the plain form


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # a short prompt of a small fp32 model: one document, two heads; latency counts
        dict(name="fwd_tiny_f32", op="fwd", T=256, lo=256, hi=256, lens=0, H=2, Hk=2, d=64,
             dtype="f32", decay="token", h0="none", scale=1.0),
        # a packed batch of documents, decay per token
        dict(name="fwd_packed", op="fwd", T=8192, lo=256, hi=2048, lens=1, H=8, Hk=8, d=128,
             dtype="bf16", decay="token", h0="none", scale=1.0),
        # one long prompt on one GPU's share of the heads
        dict(name="fwd_long", op="fwd", T=32768, lo=32768, hi=32768, lens=2, H=8, Hk=8, d=128,
             dtype="bf16", decay="token", h0="none", scale=1.0),
        # continuations of one shared prefix: ragged branches, a broadcast initial state,
        # one constant decay per head
        dict(name="fwd_branches", op="fwd", T=200000, lo=1024, hi=4096, lens=3, H=16, Hk=16, d=128,
             dtype="bf16", decay="head", h0="shared", scale=0.08838834764831845),
        # a training batch of long documents
        dict(name="bwd_train", op="bwd", T=65536, lo=4096, hi=16384, lens=4, H=8, Hk=8, d=128,
             dtype="bf16", decay="token", h0="none", scale=1.0),
        # a packed training batch with shared query/key heads, odd lengths, carried states
        dict(name="bwd_grouped_d64", op="bwd", T=8191, lo=1, hi=1500, lens=5, H=8, Hk=2, d=64,
             dtype="bf16", decay="head", h0="own", scale=0.125),
        # a small fp32 training batch (parity runs of a model in single precision)
        dict(name="bwd_f32", op="bwd", T=2047, lo=1, hi=1024, lens=6, H=4, Hk=4, d=128,
             dtype="f32", decay="token", h0="own", scale=1.0),
        # one user's next token on one GPU's share of the heads
        dict(name="step_1x8", op="step", B=1, P=4, H=8, Hk=8, d=128, dtype="bf16", decay="token",
             scale=1.0),
        # the next token of a full serving batch, states spread over a pool of pages
        dict(name="step_80x16", op="step", B=80, P=96, H=16, Hk=16, d=128, dtype="bf16",
             decay="token", scale=1.0),
        # a draft tree's small fork: last round's pages are freed, the parents fork again
        dict(name="fork_small", op="fork", P=9, parents=2, n=5, H=2, d=64),
        # a prefix state forked to a batch of branches (the prefix stays), after the last batch ended
        dict(name="fork_80", op="fork", P=96, parents=1, n=80, H=16, d=128),
        # turnover of a serving batch: finished sequences freed, the live states moved together so
        # that they form one batch again, new sequences forked from the prefix
        dict(name="turnover_128", op="turnover", P=128, n=40, H=16, d=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "fork", "turnover"])
    H = rng.choice([1, 2, 3, 4, 8, 16])
    d = rng.choice([64, 128])
    if op in ("fork", "turnover"):
        P = _log_int(rng, 4, 160)
        n = rng.randint(1, P - 2)
        if op == "turnover":
            return dict(op=op, P=P, n=n, H=H, d=d)
        return dict(op=op, P=P, parents=rng.randint(1, P - 1 - n) if P - 1 - n > 1 else 1, n=n, H=H,
                    d=d)
    Hk = rng.choice([x for x in (1, 2, 3, 4, 8, 16) if H % x == 0])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    decay = rng.choice(["token", "head"])
    scale = rng.choice([1.0, d ** -0.5])
    if op == "step":
        B = _log_int(rng, 1, 128)
        return dict(op=op, B=B, P=B + rng.randint(0, 16), H=H, Hk=Hk, d=d, dtype=dtype,
                    decay=decay, scale=scale)
    most = 65536 if op == "fwd" else 32768
    T = _log_int(rng, 1, most if dtype == "bf16" else most // 8)
    hi = _log_int(rng, 1, T)
    lo = rng.randint(0, hi)
    hi = max(hi, T // 64 + 1)  # at most a few hundred documents
    return dict(op=op, T=T, lo=lo, hi=hi, lens=rng.randint(0, 1 << 20), H=H, Hk=Hk, d=d,
                dtype=dtype, decay=decay, h0=rng.choice(["none", "own", "shared"]), scale=scale)


def lengths(case):
    """Document lengths of a case: uniform in [lo, hi] until T tokens, the last one trimmed."""
    rng, lens, left = random.Random(case["lens"] + 17), [], case["T"]
    while left > 0:
        n = min(left, rng.randint(case["lo"], case["hi"]))
        lens.append(n)
        left -= n
    return lens


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def prepare(case, seed):
    dev = _dev()
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 12345)
    normal = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    H, d = case["H"], case["d"]
    st = dict(case)
    if case["op"] in ("fork", "turnover"):
        P, n = case["P"], case["n"]
        st["pool"] = 0.5 * normal(P, H, d, d)
        order = 1 + torch.randperm(P - 1, generator=gen, device=dev).to(torch.int32)
        if case["op"] == "fork":
            # pages 0 .. are the parents and the branches of the round that has just ended
            par = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), order])[:case["parents"]]
            pick = torch.randint(case["parents"], (n,), generator=gen, device=dev)
            st["parents_of"] = par[pick].contiguous()
            st["gone"] = order[case["parents"] - 1:][:n].contiguous()
            live = torch.zeros(P, dtype=torch.int32, device=dev)
            live[par.long()] = 1
            live[st["gone"].long()] = 1
            st["live"] = live
        else:
            # every page is in use; page 0 holds the prefix; n sequences have just ended
            st["gone"] = order[:n].contiguous()
            st["parents_of"] = torch.zeros(n, dtype=torch.int32, device=dev)
            st["live"] = torch.ones(P, dtype=torch.int32, device=dev)
        return st
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    Hk = case["Hk"]
    rows = case["B"] if case["op"] == "step" else case["T"]
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    st["q"] = unit(normal(rows, Hk, d)).to(dt)
    st["k"] = unit(normal(rows, Hk, d)).to(dt)
    st["v"] = normal(rows, H, d).to(dt)
    if case["decay"] == "token":
        st["g"] = -torch.nn.functional.softplus(normal(rows, H) - 3.0)
    else:  # one horizon per head, from some 30 tokens to some thousands, moved a little by the seed
        e = -5.0 - 6.0 * torch.arange(H, device=dev) / max(1, H - 1) - 0.1 * torch.rand(
            H, generator=gen, device=dev)
        st["g"] = torch.log1p(-torch.exp2(e)).contiguous()
    if case["op"] == "step":
        st["state"] = normal(case["P"], H, d, d)
        st["pages"] = torch.randperm(case["P"], generator=gen, device=dev)[:rows].to(
            torch.int32).contiguous()
        return st
    lens = lengths(case)
    N = len(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["h0_state"] = None
    if case["h0"] != "none":
        st["h0_state"] = 0.5 * (normal(N, H, d, d) if case["h0"] == "own" else normal(H, d, d))
    if case["op"] == "bwd":
        st["dout"] = normal(rows, H, d).to(dt)
        st["dht"] = 0.5 * normal(N, H, d, d) if case["h0"] == "own" else None
    return st


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["op"]
    if own:
        import linear_attention_recurrence_prefill_amd as gdn

        if op == "fwd":
            o, ht = gdn.linattn_fwd(state["q"], state["k"], state["v"], state["g"], state["cu"],
                                    state["h0_state"], scale=state["scale"])
            return dict(o=o, ht=ht)
        if op == "bwd":
            return gdn.linattn_bwd(state["q"], state["k"], state["v"], state["g"], state["cu"],
                                   state["dout"], state["h0_state"], state["dht"],
                                   scale=state["scale"])
        if op == "step":
            o = gdn.linattn_step(state["q"], state["k"], state["v"], state["g"], state["state"],
                                 state["pages"], scale=state["scale"])
            return dict(o=o, state=state["state"])
        gdn.pages_free(state["live"], state["gone"])
        remap = gdn.pages_compact(state["pool"], state["live"]) if op == "turnover" else None
        children = gdn.pages_fork(state["pool"], state["live"], state["parents_of"])
        return dict(remap=remap, children=children, live=state["live"], pool=state["pool"])
    if op == "fwd":
        return _plain_fwd(state)
    if op == "bwd":
        return _plain_bwd(state)
    if op == "step":
        return _plain_step(state)
    return _plain_pages(state)


def _blocks(cu, T):
    """Blocks of CHUNK tokens, each within one document: (document, tokens [nc, CHUNK], valid)."""
    cu = cu.long()
    N = cu.numel() - 1
    nch = (cu[1:] - cu[:-1] + CHUNK - 1) // CHUNK
    doc = torch.repeat_interleave(torch.arange(N, device=cu.device), nch)
    nth = torch.arange(doc.numel(), device=cu.device) - (torch.cumsum(nch, 0) - nch)[doc]
    tok = (cu[doc] + CHUNK * nth)[:, None] + torch.arange(CHUNK, device=cu.device)
    valid = tok < cu[doc + 1][:, None]
    return doc, tok.clamp(max=T - 1), valid


def _take(x, tok, valid):
    """x [T, H, d] by blocks, fp32: [H, nc, CHUNK, d], rows past a document's end zero."""
    y = x[tok].float() * valid[:, :, None, None]
    return y.permute(2, 0, 1, 3).contiguous()


def _give(y, tok, valid, T, dtype):
    """The inverse of _take: [H, nc, CHUNK, d] to [T, H, d]."""
    out = torch.zeros(T, y.shape[0], y.shape[3], device=y.device, dtype=dtype)
    out[tok[valid]] = y.permute(1, 2, 0, 3)[valid].to(dtype)
    return out


def _log_decays(g, T, H, tok, valid):
    """Summed log decays within each block, 64 bits: [H, nc, CHUNK]."""
    gt = g.double() if g.dim() == 2 else g.double()[None, :].expand(T, H)
    return torch.cumsum(gt[tok].permute(2, 0, 1) * valid, -1)


def _between(doc, total, back):
    """Decay from the end of block c' to the start of block c of the same document (c' < c), or with
    `back` from the end of c to the start of c' (c' > c): [H, nc, nc], fp32."""
    end = torch.cumsum(total, -1)
    start = end - total
    diff = start[:, None, :] - end[:, :, None] if back else start[:, :, None] - end[:, None, :]
    nc = doc.numel()
    same = doc[:, None] == doc[None, :]
    order = torch.ones(nc, nc, dtype=torch.bool, device=doc.device)
    keep = same & (order.triu(1) if back else order.tril(-1))
    return torch.exp(diff.masked_fill(~keep, float("-inf")).float())


def _from_bounds(doc, total, N, back):
    """Decay from each block's document start to the block's start (or, with `back`, from the block's
    end to the document's end): [H, nc] in fp32."""
    H = total.shape[0]
    end = torch.cumsum(total, -1)
    sums = torch.zeros(H, N, dtype=torch.float64, device=total.device).index_add_(1, doc, total)
    doc_end = torch.cumsum(sums, -1)
    edge = doc_end[:, doc] if back else (doc_end - sums)[:, doc]
    return torch.exp((edge - end if back else end - total - edge).float())


def _states_of(x, N, H):
    return x if x is None or x.dim() == 4 else x[None].expand(N, *x.shape)


def _repeat(x, H):
    return x.repeat_interleave(H // x.shape[1], dim=1) if x.shape[1] != H else x


def _chunk_states(s, with_back=False):
    """What both directions share: tensors by blocks, decays, the state at each block's start."""
    v = s["v"]
    T, H, d = v.shape
    N = s["cu"].numel() - 1
    doc, tok, valid = _blocks(s["cu"], T)
    q, k, vv = (_take(_repeat(s[n], H), tok, valid) for n in ("q", "k", "v"))
    gam = _log_decays(s["g"], T, H, tok, valid)
    total = gam[..., -1]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    dec = torch.exp((gam[..., :, None] - gam[..., None, :]).masked_fill(~low, float("-inf")).float())
    f_in = torch.exp(gam.float())[..., None]
    f_end = torch.exp((total[..., None] - gam).float())[..., None]
    nc = doc.numel()
    local = (k * f_end).transpose(-1, -2) @ vv
    S0 = (_between(doc, total, False) @ local.reshape(H, nc, d * d)).reshape(H, nc, d, d)
    h0 = _states_of(s["h0_state"], N, H)
    if h0 is not None:
        S0 = S0 + _from_bounds(doc, total, N, False)[..., None, None] * h0[doc].transpose(0, 1)
    return dict(T=T, H=H, d=d, N=N, doc=doc, tok=tok, valid=valid, q=q, k=k, v=vv, gam=gam,
                total=total, dec=dec, f_in=f_in, f_end=f_end, local=local, S0=S0, h0=h0)


def _edge_states(at, doc, per_block, N, other):
    """Per document the state of its last (at=-1) or first (at=0) block; `other` (or zero) where a
    document has no block."""
    H, nc, d = per_block.shape[0], per_block.shape[1], per_block.shape[2]
    out = torch.zeros(N, H, d, d, device=per_block.device) if other is None else other.clone()
    edge = torch.ones(nc, dtype=torch.bool, device=doc.device)
    if at == -1:
        edge[:-1] = doc[1:] != doc[:-1]
    else:
        edge[1:] = doc[1:] != doc[:-1]
    out[doc[edge]] = per_block[:, edge].transpose(0, 1)
    return out


def _plain_fwd(s):
    c = _chunk_states(s)
    att = (c["q"] @ c["k"].transpose(-1, -2)) * c["dec"]
    o = s["scale"] * (c["f_in"] * (c["q"] @ c["S0"]) + att @ c["v"])
    S1 = torch.exp(c["total"].float())[..., None, None] * c["S0"] + c["local"]
    ht = _edge_states(-1, c["doc"], S1, c["N"], c["h0"])
    return dict(o=_give(o, c["tok"], c["valid"], c["T"], s["v"].dtype), ht=ht)


def _plain_bwd(s):
    c = _chunk_states(s)
    T, H, d, N, doc, total = c["T"], c["H"], c["d"], c["N"], c["doc"], c["total"]
    tok, valid, q, k, v, S0, scale = c["tok"], c["valid"], c["q"], c["k"], c["v"], c["S0"], s["scale"]
    nc = doc.numel()
    do = _take(s["dout"], tok, valid)
    back = scale * (q.transpose(-1, -2) @ (c["f_in"] * do))
    dS = (_between(doc, total, True) @ back.reshape(H, nc, d * d)).reshape(H, nc, d, d)
    if s["dht"] is not None:
        dS = dS + _from_bounds(doc, total, N, True)[..., None, None] * s["dht"][doc].transpose(0, 1)
    qk, dov = q @ k.transpose(-1, -2), do @ v.transpose(-1, -2)
    att, datt = scale * qk * c["dec"], scale * dov * c["dec"]
    dq_in = scale * c["f_in"] * (do @ S0.transpose(-1, -2))
    dk_in = c["f_end"] * (v @ dS.transpose(-1, -2))
    dq = dq_in + datt @ k
    dk = dk_in + datt.transpose(-1, -2) @ q
    dv = c["f_end"] * (k @ dS) + att.transpose(-1, -2) @ do
    # dg_t = <dS_t, exp(g_t) S_{t-1}>: pairs within the block on both sides of t, the block's
    # queries with its start state, its keys with its end gradient, and both states
    strict = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril(-1)
    pairs = (att * dov).masked_fill(~strict, 0.0).double()
    pairs = pairs.flip(-2).cumsum(-2).flip(-2).masked_fill(~strict, 0.0).sum(-1)
    qi, ki = (q * dq_in).double().sum(-1), (k * dk_in).double().sum(-1)
    both = torch.exp(total) * (dS * S0).double().sum((-1, -2))
    dg = pairs + qi.flip(-1).cumsum(-1).flip(-1) + ki.cumsum(-1) - ki + both[..., None]
    dgt = torch.zeros(T, H, dtype=torch.float64, device=q.device)
    dgt[tok[valid]] = dg.permute(1, 2, 0)[valid]
    dg = (dgt if s["g"].dim() == 2 else dgt.sum(0)).float()
    dh0 = torch.exp(total.float())[..., None, None] * dS + back
    dh0 = _edge_states(0, doc, dh0, N, s["dht"])
    if s["h0_state"] is not None and s["h0_state"].dim() == 3:
        dh0 = dh0.double().sum(0).float()
    Hk = s["q"].shape[1]
    if Hk != H:
        dq, dk = (x.reshape(Hk, H // Hk, nc, CHUNK, d).sum(1) for x in (dq, dk))
    give = lambda y: _give(y, tok, valid, T, s["v"].dtype)  # noqa: E731
    return dict(dq=give(dq), dk=give(dk), dv=give(dv), dg=dg, dh0=dh0)


def _plain_step(s):
    H = s["v"].shape[1]
    q, k, v = _repeat(s["q"], H).float(), _repeat(s["k"], H).float(), s["v"].float()
    pages = s["pages"].long()
    g = s["g"] if s["g"].dim() == 2 else s["g"][None].expand(v.shape[0], H)
    S = torch.exp(g)[..., None, None] * s["state"][pages] + k[..., :, None] * v[..., None, :]
    s["state"][pages] = S
    o = s["scale"] * (q[..., :, None] * S).sum(-2)
    return dict(o=o.to(s["v"].dtype), state=s["state"])


def _plain_pages(s):
    pool, live = s["pool"], s["live"]
    live[s["gone"].long()] = 0
    remap = None
    if s["op"] == "turnover":
        used = live != 0
        count = used.sum()
        place = torch.arange(live.numel(), device=live.device)
        holes, movers = place[~used & (place < count)], place[used & (place >= count)]
        new = place.clone()
        new[movers] = holes
        remap = torch.where(used, new, -1).to(torch.int32)
        pool[holes] = pool[movers]
        live.copy_((place < count).to(torch.int32))
    children = torch.nonzero(live == 0)[:s["parents_of"].numel(), 0]
    pool[children] = pool[s["parents_of"].long()]
    live[children] = 1
    return dict(remap=remap, children=children.to(torch.int32), live=live, pool=pool)


# ---------------------------------------------------------------------------------------------
# cost
# ---------------------------------------------------------------------------------------------

def work(case):
    H, d = case["H"], case["d"]
    page = 4.0 * H * d * d
    if case["op"] == "fork":
        return dict(bytes=page * (case["parents"] + case["n"]), flops=0.0)
    if case["op"] == "turnover":  # expected moves: the ended sequences among the pages that stay
        moves = case["n"] * (case["P"] - case["n"]) / case["P"]
        return dict(bytes=page * (2 * moves + 1 + case["n"]), flops=0.0)
    es = 2 if case["dtype"] == "bf16" else 4
    Hk = case["Hk"]
    if case["op"] == "step":
        B = case["B"]
        return dict(bytes=2.0 * page * B + B * d * es * 2.0 * (Hk + H) + 4.0 * B * H,
                    flops=5.0 * B * H * d * d)
    T, N = case["T"], len(lengths(case))
    g = 4.0 * H * (T if case["decay"] == "token" else 1)
    states = {"none": 0, "own": N, "shared": 1}[case["h0"]]
    if case["op"] == "fwd":
        return dict(bytes=T * d * es * 2.0 * (Hk + H) + g + page * (states + N),
                    flops=4.0 * T * H * d * d)
    dh0 = 1 if case["h0"] == "shared" else N
    dht = N if case["h0"] == "own" else 0
    return dict(bytes=T * d * es * (4.0 * Hk + 3.0 * H) + 2 * g + page * (states + dh0 + dht),
                flops=10.0 * T * H * d * d)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits: token by token, every document and head side by side
# ---------------------------------------------------------------------------------------------

def _padded(x, cu, longest):
    """[T, H, ...] to [longest, N, H, ...], 64 bits, zero past each document's end."""
    at = cu[:-1].long()[None, :] + torch.arange(longest, device=x.device)[:, None]
    inside = at < cu[1:].long()[None, :]
    y = x.double()[at.clamp(max=x.shape[0] - 1)]
    return y * inside.reshape(*inside.shape, *([1] * (y.dim() - 2))), at, inside


def exact(case, seed):
    s = prepare(case, seed)
    op, H, d = case["op"], case["H"], case["d"]
    if op in ("fork", "turnover"):
        pool, live = s["pool"].double(), s["live"].tolist()
        for p in s["gone"].tolist():
            live[p] = 0
        remap = None
        if op == "turnover":
            count = sum(live)
            remap, movers = [-1] * len(live), [p for p in range(count, len(live)) if live[p]]
            for p in range(len(live)):
                if live[p] and p < count:
                    remap[p] = p
            for p in range(count):
                if not live[p]:
                    frm = movers.pop(0)
                    remap[frm] = p
                    pool[p] = pool[frm].clone()
            live = [1] * count + [0] * (len(live) - count)
            remap = torch.tensor(remap, dtype=torch.int32)
        children = []
        for parent in s["parents_of"].tolist():
            child = live.index(0)
            pool[child] = pool[parent].clone()
            live[child] = 1
            children.append(child)
        return dict(remap=remap, children=torch.tensor(children, dtype=torch.int32),
                    live=torch.tensor(live, dtype=torch.int32), pool=pool)
    rep = H // case["Hk"]
    wide = lambda x: x.repeat_interleave(rep, dim=1)  # noqa: E731
    if op == "step":
        state = s["state"].double()
        q, k, v = wide(s["q"].double()), wide(s["k"].double()), s["v"].double()
        o = torch.empty_like(v)
        for b, p in enumerate(s["pages"].tolist()):
            g = s["g"].double() if s["g"].dim() == 1 else s["g"][b].double()
            state[p] = state[p] * g.exp()[:, None, None] + k[b][:, :, None] * v[b][:, None, :]
            o[b] = s["scale"] * torch.einsum("hk,hkv->hv", q[b], state[p])
        return dict(o=o, state=state)
    T, cu = case["T"], s["cu"]
    N, longest = cu.numel() - 1, max(lengths(case))
    if longest * N * H * d > 1.5e9 or longest * N * H * d * d > 3e11:
        return None  # padded to its longest document this takes too much memory or time
    names = ("q", "k", "v") + (("dout",) if op == "bwd" else ())
    t = {}
    for n in names:
        x = wide(s[n]) if n in ("q", "k") else s[n]
        t[n], at, inside = _padded(x, cu, longest)
    g = s["g"] if s["g"].dim() == 2 else s["g"][None].expand(T, H)
    a = _padded(g, cu, longest)[0].exp()[..., None, None]  # exp(0) = 1 past a document's end
    h0 = s["h0_state"]
    S = torch.zeros(N, H, d, d, dtype=torch.float64, device=cu.device) if h0 is None else \
        (h0.double() if h0.dim() == 4 else h0.double()[None].expand(N, H, d, d)).clone()
    k4, v4 = t["k"][..., :, None], t["v"][..., None, :]
    back = lambda y: _unpad(y, at, inside, T)  # noqa: E731
    if op == "fwd":
        o = torch.empty_like(t["v"])
        for i in range(longest):
            S = S * a[i] + k4[i] * v4[i]
            o[i] = s["scale"] * (t["q"][i][..., :, None] * S).sum(-2)
        return dict(o=back(o), ht=S)
    dq, dk, dv = (torch.empty_like(t["v"]) for _ in range(3))
    for i in range(longest):
        S = S * a[i] + k4[i] * v4[i]
        dq[i] = s["scale"] * (S * t["dout"][i][..., None, :]).sum(-1)
    dht = s["dht"]
    dS = torch.zeros_like(S) if dht is None else dht.double()
    end = (dS * S).sum((-1, -2))
    for i in range(longest - 1, -1, -1):
        dS = dS + s["scale"] * t["q"][i][..., :, None] * t["dout"][i][..., None, :]
        dk[i] = (dS * v4[i]).sum(-1)
        dv[i] = (dS * k4[i]).sum(-2)
        dS = dS * a[i]
    # each log decay scales everything that crosses it: what later queries read of earlier keys
    cross = (t["q"] * dq).sum(-1) - (t["k"] * dk).sum(-1)
    dg = back((cross.flip(0).cumsum(0).flip(0) + end)[..., None])[..., 0]
    if rep > 1:
        dq, dk = (x.reshape(longest, N, case["Hk"], rep, d).sum(3) for x in (dq, dk))
    return dict(dq=back(dq), dk=back(dk), dv=back(dv), dg=dg if s["g"].dim() == 2 else dg.sum(0),
                dh0=dS.sum(0) if h0 is not None and h0.dim() == 3 else dS)


def _unpad(y, at, inside, T):
    out = torch.zeros(T, *y.shape[2:], dtype=y.dtype, device=y.device)
    out[at[inside]] = y[inside]
    return out
