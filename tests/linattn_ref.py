"""Linear attention with a decay for each head in 64 bits on the CPU, token by token, for the tests:
the definition itself, with gradients by autograd.  Shares nothing with the library."""
import torch


def forward(q, k, v, g, cu, h0=None, scale=1.0):
    """q, k [T, Hk, D], v [T, H, D], g [T, H] or [H], h0 None, [N, H, D, D] or [H, D, D]: (o, ht)."""
    T, H, D = v.shape
    q, k = (x.repeat_interleave(H // x.shape[1], dim=1) for x in (q, k))
    if g.dim() == 1:
        g = g[None].expand(T, H)
    outs, states = [], []
    for n in range(len(cu) - 1):
        if h0 is None:
            S = torch.zeros(H, D, D, dtype=torch.float64)
        else:
            S = h0 if h0.dim() == 3 else h0[n]
        for t in range(int(cu[n]), int(cu[n + 1])):
            S = torch.exp(g[t])[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            outs.append(scale * (q[t][:, :, None] * S).sum(1))
        states.append(S)
    o = torch.stack(outs) if outs else torch.zeros(0, H, D, dtype=torch.float64)
    return o, torch.stack(states)


def backward(q, k, v, g, cu, dout, h0=None, dht=None, scale=1.0):
    """Gradients of <o, dout> + <ht, dht>: dict(dq, dk, dv, dg, dh0) (dh0 per h0's shape, per
    sequence when h0 is None)."""
    H, D = v.shape[1:]
    ins = [x.double().clone().requires_grad_() for x in (q, k, v, g)]
    start = torch.zeros(len(cu) - 1, H, D, D, dtype=torch.float64) if h0 is None else h0.double()
    start = start.clone().requires_grad_()
    o, ht = forward(*ins, cu, start, scale)
    loss = (o * dout.double()).sum() + (0 if dht is None else (ht * dht.double()).sum())
    grads = torch.autograd.grad(loss, ins + [start], allow_unused=True)
    zero = lambda x, gr: torch.zeros_like(x) if gr is None else gr  # noqa: E731
    return {n: zero(x, gr) for n, x, gr in zip(("dq", "dk", "dv", "dg", "dh0"), ins + [start], grads)}


def inputs(lens, H, Hk, D, dtype, decay="token", h0="none", dht=False, seed=0, g_mu=-3.0):
    """Seeded tensors on the CPU in the library's types: q and k rows of unit length, v and dout
    normal, g = -softplus(N(g_mu, 1))."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    T, N = sum(lens), len(lens)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    g = -torch.nn.functional.softplus(rand(T, H) + g_mu if decay == "token" else rand(H) + g_mu)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return dict(q=unit(rand(T, Hk, D)).to(dt), k=unit(rand(T, Hk, D)).to(dt),
                v=rand(T, H, D).to(dt), g=g.float(), cu=torch.tensor(cu, dtype=torch.int32),
                dout=rand(T, H, D).to(dt),
                h0={"none": None, "own": 0.5 * rand(N, H, D, D),
                    "shared": 0.5 * rand(H, D, D)}[h0],
                dht=0.5 * rand(N, H, D, D) if dht else None)


def to64(x):
    return None if x is None else x.detach().double().cpu()


def rel(x, ref):
    """Relative L2 distance in 64 bits (absolute where ref is zero)."""
    x, ref = to64(x), to64(ref)
    den = ref.norm()
    return float((x - ref).norm() / (den if den > 0 else 1.0))
