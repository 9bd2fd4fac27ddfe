"""Linear attention with a decay for each head on the GPU against its definition in 64 bits
(tests/linattn_ref.py, gradients by autograd; gfx950 only; marked ``gpu``).

Tolerances, as relative L2 over a tensor.  bf16 outputs carry one rounding of at most 2^-8 of each
value, rho = 2^-8 / sqrt 3 in the mean square.  o and dv of units longer than four chunks also carry
the one rounding of the state that they read, elementwise and independent, so rho of the part from
the state; two such roundings add to sqrt(2) rho < 2^-8.  Everything else before the output is held to
2^-16 (operands split into two bf16 terms) or better, so 2^-8 + 2^-12 bounds the distance.  fp32 results are sums: each addition or product rounds by at most
u = 2^-24, and an element of these cases passes through at most some 10^3 of them (64-token chunks
summed by 16-term products, one decay and one addition of the state per chunk, the D-term products)
whose errors are independent, so sqrt(10^3) u = 2e-6; F32_TOL = 4e-6 is twice that.  dg also
cancels: it is a difference of sums of |q . dq| and |k . dk| over up to a unit's tokens, held to
2e-5 (the same count for the two sums, an order of magnitude for the cancellation)."""
import ctypes
import itertools

import pytest

torch = pytest.importorskip("torch")

import linattn_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BF16_TOL, F32_TOL, DG_TOL = 2.0 ** -8 + 2.0 ** -12, 4e-6, 2e-5


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_attention_recurrence_prefill_amd as m

    m.load_library()
    return m


def dev(x, device="cuda"):
    return {n: None if t is None else (t.float() if n in ("h0", "dht") else t).to(device)
            for n, t in x.items()}


def host64(x):
    """The library's inputs as the reference takes them (the rounded values)."""
    return {n: None if t is None else (t if n == "cu" else t.float().double())
            for n, t in x.items()}


def check(name, got, want, tol):
    err = ref.rel(got, want)
    print(f"  {name}: {err:.2e} (tol {tol:.1e})", flush=True)
    assert torch.isfinite(got.float()).all(), name
    assert err <= tol, f"{name}: {err:.3e} > {tol:.1e}"


def tols(dtype):
    t = BF16_TOL if dtype == "bf16" else F32_TOL
    return dict(o=t, ht=F32_TOL, dq=t, dk=t, dv=t, dg=DG_TOL, dh0=F32_TOL)


def run_both(gdn, x, dtype, scale=1.0, what=("fwd", "bwd"), **kw):
    d, r, tol = dev(x), host64(x), tols(dtype)
    args = [d[n] for n in ("q", "k", "v", "g", "cu")]
    rargs = [r[n] for n in ("q", "k", "v", "g", "cu")]
    if "fwd" in what:
        o, ht = gdn.linattn_fwd(*args, d["h0"], scale=scale, **kw)
        torch.cuda.synchronize()
        o_ref, ht_ref = ref.forward(*rargs, r["h0"], scale)
        check("o", o, o_ref, tol["o"])
        check("ht", ht, ht_ref, tol["ht"])
    if "bwd" in what:
        got = gdn.linattn_bwd(*args, d["dout"], d["h0"], d["dht"], scale=scale, **kw)
        torch.cuda.synchronize()
        want = ref.backward(*rargs, r["dout"], r["h0"], r["dht"], scale)
        for n in want:
            check(n, got[n], want[n], tol[n])


LENS = [1, 0, 63, 64, 65, 130, 0, 17]


@pytest.mark.parametrize("dtype,D", itertools.product(("bf16", "f32"), (64, 128)))
@pytest.mark.parametrize("decay,h0,dht,H,Hk,seg", [
    ("token", "none", False, 2, 2, 0), ("head", "own", True, 4, 2, 0),
    ("token", "shared", True, 3, 1, 1), ("head", "shared", False, 2, 2, 2)])
def test_forward_and_backward(gdn, dtype, D, decay, h0, dht, H, Hk, seg):
    x = ref.inputs(LENS, H, Hk, D, dtype, decay, h0, dht, seed=11)
    run_both(gdn, x, dtype, 0.7, seg_chunks=seg)


@pytest.mark.parametrize("dtype,D,seg", [("bf16", 128, 0), ("bf16", 128, 3), ("bf16", 64, 2),
                                         ("f32", 64, 3), ("f32", 128, 4)])
def test_long_sequences_in_units(gdn, dtype, D, seg):
    """Documents of many units, with a ragged end, and one unit exactly full."""
    x = ref.inputs([64 * 6, 701, 5], 2, 1, D, dtype, "token", "own", True, seed=12)
    run_both(gdn, x, dtype, 1.0, seg_chunks=seg)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,seg", [([450, 70], 0), ([450, 70], 2), ([450, 70], 1000), ([130, 0, 1], 1)])
def test_many_heads(gdn, lens, seg, D):
    """More workgroups than CUs in every stage: two heads of the reference, 140 times over."""
    x = ref.inputs(lens, 2, 2, D, "bf16", "token", "own", True, seed=22)
    r, tol = host64(x), tols("bf16")
    rargs = [r[n] for n in ("q", "k", "v", "g", "cu")]
    o_ref, ht_ref = ref.forward(*rargs, r["h0"], 0.5)
    want = ref.backward(*rargs, r["dout"], r["h0"], r["dht"], 0.5)
    many = lambda t: t.repeat(*(140 if i == 1 else 1 for i in range(t.dim())))  # noqa: E731
    d = dev({n: t if n == "cu" else many(t) for n, t in x.items()})
    args = [d[n] for n in ("q", "k", "v", "g", "cu")]
    o, ht = gdn.linattn_fwd(*args, d["h0"], scale=0.5, seg_chunks=seg)
    check("o", o, many(o_ref), tol["o"])
    check("ht", ht, many(ht_ref), tol["ht"])
    got = gdn.linattn_bwd(*args, d["dout"], d["h0"], d["dht"], scale=0.5, seg_chunks=seg)
    for n in want:
        check(n, got[n], many(want[n]), tol[n])


@pytest.mark.parametrize("Hk", [4, 2])
@pytest.mark.parametrize("seg", [1, 1000])
def test_rows_of_no_sequence_stay(gdn, Hk, seg):
    """Tokens after the last sequence: outputs there are left as they were, and NaN in their inputs
    reaches nothing."""
    x = ref.inputs([70, 100], 4, Hk, 64, "bf16", "token", "none", False, seed=23)
    pad = lambda t: torch.cat([t, torch.full_like(t[:9], float("nan"))])  # noqa: E731
    d = dev(x)
    names = ("q", "k", "v", "g", "dout")
    w = {n: pad(d[n]) for n in names}
    cu = d["cu"]
    o, ht = gdn.linattn_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], seg_chunks=seg)
    got = gdn.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["dout"], seg_chunks=seg)
    out = torch.full_like(w["v"], 7.0)
    o2, ht2 = gdn.linattn_fwd(w["q"], w["k"], w["v"], w["g"], cu, out=out, seg_chunks=seg)
    assert torch.equal(o2[:170], o) and torch.equal(ht2, ht)
    assert (o2[170:] == 7).all()
    lib = gdn.load_library()
    from linear_attention_recurrence_prefill_amd.linattn import _at, _problem

    p, device, N, H, D = _problem(w["q"], w["k"], w["v"], w["g"], cu, None, 1.0, seg, 0)
    res = {"d" + n: torch.full_like(w[n], 7.0) for n in ("q", "k", "v", "g")}
    dh0 = torch.empty(N, H, D, D, device=device)
    ws = torch.empty(gdn.gdn_linattn_bwd_workspace_size(w["q"], w["k"], w["v"], w["g"], cu, seg_chunks=seg),
                     dtype=torch.uint8, device=device)
    status = lib.gdn_linattn_bwd(ctypes.byref(p), *(_at(w[n]) for n in ("q", "k", "v", "g")), _at(cu),
                                 None, _at(w["dout"]), None,
                                 *(_at(res[n]) for n in ("dq", "dk", "dv", "dg")), _at(dh0), _at(ws),
                                 ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0 and torch.equal(dh0, got["dh0"])
    for n, t in res.items():
        assert torch.equal(t[:170], got[n]), n
        assert (t[170:] == 7).all(), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 48, 63, 127])
def test_short_documents(gdn, dtype, T):
    x = ref.inputs([T], 2, 2, 128, dtype, "token", "own", True, seed=100 + T)
    run_both(gdn, x, dtype, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "strong", "reset", "mixed"])
def test_decays_at_the_edges(gdn, dtype, kind):
    """No decay at all, decays of e^-5 per token, states emptied by -inf, and a reset between tokens
    that hardly decay.  A reset's own gradient is zero; with strong decays dg is of order e^-5 of
    the products it is summed from, so it is compared on their scale."""
    x = ref.inputs([150, 64, 70], 2, 2, 128, dtype, "token", "own", True, seed=13)
    g = x["g"]
    if kind == "none":
        g.zero_()
    elif kind == "strong":
        g.sub_(5.0)
    elif kind == "reset":
        g[::7] = float("-inf")
    else:
        g.mul_(0.01)
        g[40], g[41], g[100] = -60.0, -300.0, -1e30
    d, r, tol = dev(x), host64(x), tols(dtype)
    args = [d[n] for n in ("q", "k", "v", "g", "cu")]
    o, ht = gdn.linattn_fwd(*args, d["h0"], seg_chunks=1)
    got = gdn.linattn_bwd(*args, d["dout"], d["h0"], d["dht"], seg_chunks=1)
    torch.cuda.synchronize()
    # the definition with exp(-inf) = 0; autograd through exp gives a zero gradient there
    rargs = [r[n].clamp(min=-1e4) if n == "g" else r[n] for n in ("q", "k", "v", "g", "cu")]
    o_ref, ht_ref = ref.forward(*rargs, r["h0"])
    want = ref.backward(*rargs, r["dout"], r["h0"], r["dht"])
    check("o", o, o_ref, tol["o"])
    check("ht", ht, ht_ref, tol["ht"])
    for n in ("dq", "dk", "dv", "dh0"):
        check(n, got[n], want[n], tol[n])
    terms = (r["q"] * want["dq"]).sum(-1).norm() + (r["k"] * want["dk"]).sum(-1).norm()
    err = float((got["dg"].double().cpu() - want["dg"]).norm() / terms)
    print(f"  dg: {err:.2e}", flush=True)
    assert err <= F32_TOL
    assert (got["dg"].cpu()[x["g"] < -110] == 0).all()


def test_split_and_whole_sequences_agree(gdn):
    """The split is exact: the same numbers up to rounding, whatever the units' length."""
    x = dev(ref.inputs([900, 333], 3, 3, 128, "bf16", "token", "own", True, seed=14))
    args = [x[n] for n in ("q", "k", "v", "g", "cu")]
    whole = gdn.linattn_fwd(*args, x["h0"], seg_chunks=1000)
    gw = gdn.linattn_bwd(*args, x["dout"], x["h0"], x["dht"], seg_chunks=1000)
    for seg in (1, 2, 5, 14):
        o, ht = gdn.linattn_fwd(*args, x["h0"], seg_chunks=seg)
        got = gdn.linattn_bwd(*args, x["dout"], x["h0"], x["dht"], seg_chunks=seg)
        # o and dv of long units round the state's elements to bf16, and of short units not: the two
        # results differ by that rounding, at most 2^-8 of each element, rho = 2^-8 / sqrt 3 in the
        # mean square and independent from element to element, so rho of the sum over the state's
        # rows; and by the two roundings of the results, each rho again: sqrt(3) rho = 2^-8
        assert ref.rel(o, whole[0]) <= 2.0 ** -8
        assert ref.rel(got["dv"], gw["dv"]) <= 2.0 ** -8
        assert ref.rel(ht, whole[1]) <= F32_TOL
        assert ref.rel(got["dg"], gw["dg"]) <= DG_TOL
        assert ref.rel(got["dh0"], gw["dh0"]) <= F32_TOL
        # these differ where a last fp32 bit tips the rounding: by one step of 2^-8, rarely
        assert all(ref.rel(got[n], gw[n]) <= 2.0 ** -10 for n in ("dq", "dk"))


def test_no_tokens(gdn):
    """Every sequence empty: states pass through, and nothing else is written."""
    e = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    h0 = torch.randn(3, 2, 64, 64, device="cuda")
    g = torch.empty(0, 2, device="cuda")
    o, ht = gdn.linattn_fwd(e, e, e, g, cu, h0)
    assert o.shape == (0, 2, 64) and torch.equal(ht, h0)
    assert torch.equal(gdn.linattn_fwd(e, e, e, g, cu)[1], torch.zeros_like(h0))
    got = gdn.linattn_bwd(e, e, e, torch.zeros(2, device="cuda"), cu, e, h0, h0)
    assert torch.equal(got["dh0"], h0) and torch.equal(got["dg"], torch.zeros(2, device="cuda"))
    got = gdn.linattn_bwd(e, e, e, g, cu, e, h0[0].contiguous(), h0)
    assert ref.rel(got["dh0"], h0.double().sum(0)) <= F32_TOL


def test_sequences_do_not_mix_and_results_repeat(gdn):
    """Bitwise: the same call twice, and other documents' results when one document changes."""
    x = dev(ref.inputs([200, 129, 300], 4, 2, 128, "bf16", "token", "none", False, seed=15))
    y = dict(x)
    for n in ("q", "k", "v", "g", "dout"):
        y[n] = x[n].clone()
        y[n][200:329] *= 0.5
    run = lambda z: (gdn.linattn_fwd(*[z[n] for n in ("q", "k", "v", "g", "cu")], seg_chunks=2),  # noqa: E731
                     gdn.linattn_bwd(*[z[n] for n in ("q", "k", "v", "g", "cu")], z["dout"], seg_chunks=2))
    (o1, h1), b1 = run(x)
    (o2, h2), b2 = run(x)
    assert torch.equal(o1, o2) and torch.equal(h1, h2)
    assert all(torch.equal(b1[n], b2[n]) for n in b1)
    (o3, h3), b3 = run(y)
    rest = torch.ones(629, dtype=torch.bool, device="cuda")
    rest[200:329] = False
    assert torch.equal(o1[rest], o3[rest]) and not torch.equal(o1[~rest], o3[~rest])
    assert torch.equal(h1[0], h3[0]) and torch.equal(h1[2], h3[2])
    assert all(torch.equal(b1[n][rest], b3[n][rest]) for n in ("dq", "dk", "dv", "dg"))


def test_non_finite_token_stays_in_its_sequence(gdn):
    """A NaN token: other sequences and heads, and its own sequence's earlier chunks, are as they
    would be without it."""
    x = dev(ref.inputs([200, 129, 300], 2, 2, 128, "bf16", "token", "none", False, seed=16))
    args = [x[n] for n in ("q", "k", "v", "g", "cu")]
    o1, h1 = gdn.linattn_fwd(*args, seg_chunks=2)
    x["v"][200 + 70, 1, 3] = float("nan")
    o2, h2 = gdn.linattn_fwd(*args, seg_chunks=2)
    hit = torch.zeros(629, 2, dtype=torch.bool, device="cuda")
    hit[200 + 64:329, 1] = True
    assert torch.equal(o1[~hit], o2[~hit])
    assert torch.equal(h1[:, 0], h2[:, 0]) and torch.equal(h1[::2], h2[::2])
    assert torch.isnan(o2[200 + 70:329, 1, 3].float()).all() and torch.isnan(h2[1, 1, :, 3]).all()


def test_writes_only_its_outputs(gdn):
    """Outputs and workspace inside larger buffers of sentinels: nothing around them changes."""
    x = dev(ref.inputs([70, 65], 2, 2, 128, "bf16", "token", "own", True, seed=17))
    args = [x[n] for n in ("q", "k", "v", "g", "cu")]
    pad = 4096

    def guarded(shape, dtype):
        n = 1
        for s in shape:
            n *= s
        buf = torch.full((n + 2 * pad,), 7.0, device="cuda").to(dtype)
        return buf, buf[pad:pad + n].view(shape)

    bo, o = guarded((135, 2, 128), torch.bfloat16)
    bh, ht = guarded((2, 2, 128, 128), torch.float32)
    from linear_attention_recurrence_prefill_amd import linattn

    need = linattn.linattn_fwd_workspace_bytes(*args, x["h0"], seg_chunks=1)
    bw, ws = guarded((need,), torch.uint8)
    gdn.linattn_fwd(*args, x["h0"], seg_chunks=1, out=o, final_state=ht, workspace=ws)
    torch.cuda.synchronize()
    for b in (bo, bh, bw):
        assert (b[:pad] == 7).all() and (b[-pad:] == 7).all()
    o2, h2 = gdn.linattn_fwd(*args, x["h0"], seg_chunks=1)
    assert torch.equal(o, o2) and torch.equal(ht, h2)
    need = linattn.linattn_bwd_workspace_bytes(*args, x["h0"], seg_chunks=1)
    bw, ws = guarded((need,), torch.uint8)
    gdn.linattn_bwd(*args, x["dout"], x["h0"], x["dht"], seg_chunks=1, workspace=ws)
    torch.cuda.synchronize()
    assert (bw[:pad] == 7).all() and (bw[-pad:] == 7).all()


# ---- one token -----------------------------------------------------------------------------------

def step_inputs(B, H, Hk, D, dtype, decay, seed, extra=0):
    x = ref.inputs([1] * B, H, Hk, D, dtype, decay, "none", False, seed=seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x["state"] = torch.randn(B + extra, H, D, D, generator=gen)
    x["pages"] = torch.randperm(B + extra, generator=gen)[:B].to(torch.int32)
    return x


def step_ref(x, rows, scale):
    """(o, new states) of the given rows, each on the state of its page."""
    r = host64(x)
    H = r["v"].shape[1]
    g = r["g"] if r["g"].dim() == 2 else r["g"][None].expand(r["v"].shape[0], H)
    rep = H // r["q"].shape[1]
    q, k = (r[n].repeat_interleave(rep, dim=1)[rows] for n in ("q", "k"))
    S = x["state"].double()[x["pages"].long()[rows]]
    S = g[rows].exp()[..., None, None] * S + k[..., :, None] * r["v"][rows][..., None, :]
    return scale * (q[..., :, None] * S).sum(-2), S


@pytest.mark.parametrize("dtype,D", itertools.product(("bf16", "f32"), (64, 128)))
@pytest.mark.parametrize("decay,Hk", [("token", 4), ("head", 2)])
def test_step_on_pages(gdn, dtype, D, decay, Hk):
    B, H = 7, 4
    x = step_inputs(B, H, Hk, D, dtype, decay, 21, extra=5)
    d = dev(x)
    before = d["state"].clone()
    o = gdn.linattn_step(d["q"], d["k"], d["v"], d["g"], d["state"], d["pages"], scale=0.6)
    torch.cuda.synchronize()
    o_ref, S_ref = step_ref(x, slice(None), 0.6)
    check("o", o, o_ref, BF16_TOL if dtype == "bf16" else F32_TOL)
    check("state", d["state"][d["pages"].long()], S_ref, F32_TOL)
    other = torch.ones(B + 5, dtype=torch.bool, device="cuda")
    other[d["pages"].long()] = False
    assert torch.equal(d["state"][other], before[other])


def test_step_on_a_plain_batch_equals_pages(gdn):
    x = dev(step_inputs(5, 3, 1, 128, "bf16", "token", 22))
    s1, s2 = x["state"].clone(), x["state"].clone()
    o1 = gdn.linattn_step(x["q"], x["k"], x["v"], x["g"], s1)
    o2 = gdn.linattn_step(x["q"], x["k"], x["v"], x["g"], s2,
                          torch.arange(5, dtype=torch.int32, device="cuda"))
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


def test_step_rows_without_a_page(gdn):
    """Padding (-1), pages outside the pool and a page named twice: zeros out, no state touched but
    the first row's; all but padding are reported."""
    x = step_inputs(6, 2, 2, 64, "bf16", "token", 23, extra=4)
    d = dev(x)
    pages = d["pages"].clone()
    pages[1], pages[2], pages[3], pages[5] = -1, 10, -7, pages[0]
    before = d["state"].clone()
    gdn.device_faults(clear=True)
    o = gdn.linattn_step(d["q"], d["k"], d["v"], d["g"], d["state"], pages)
    torch.cuda.synchronize()
    o_ref, S_ref = step_ref(x, [0, 4], 1.0)
    check("o", o[[0, 4]], o_ref, BF16_TOL)
    check("state", d["state"][pages[[0, 4]].long()], S_ref, F32_TOL)
    assert (o[[1, 2, 3, 5]] == 0).all()
    other = torch.ones(10, dtype=torch.bool, device="cuda")
    other[pages[[0, 4]].long()] = False
    assert torch.equal(d["state"][other], before[other])
    assert gdn.device_faults(clear=True) == 2 | 4
    pages[:] = -1
    before = d["state"].clone()
    o = gdn.linattn_step(d["q"], d["k"], d["v"], d["g"], d["state"], pages)
    assert (o == 0).all() and torch.equal(d["state"], before) and gdn.device_faults() == 0


def test_prefill_then_steps_equal_one_longer_sequence(gdn):
    """A prompt by chunks, its states put into pages, then tokens one by one: the recurrence over all
    of them."""
    B, H, D, n, extra = 3, 2, 128, 100, 8
    x = ref.inputs([n + extra] * B, H, H, D, "bf16", "token", seed=24)
    d, r = dev(x), host64(x)
    rows = torch.arange(B * (n + extra)).view(B, n + extra)
    cut = lambda m, t: m[t[:, :n].reshape(-1)].contiguous()  # noqa: E731
    pre = [cut(d[m], rows.cuda()) for m in ("q", "k", "v", "g")]
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    _, ht = gdn.linattn_fwd(*pre, cu)
    pool = torch.full((6, H, D, D), float("nan"), device="cuda")
    pages = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    gdn.pages_copy(pool, ht, pages, torch.arange(B, dtype=torch.int32, device="cuda"))
    outs = []
    for s in range(extra):
        at = rows[:, n + s].cuda()
        outs.append(gdn.linattn_step(*[d[m][at].contiguous() for m in ("q", "k", "v", "g")], pool,
                                     pages))
    o_ref, ht_ref = ref.forward(*[r[m] for m in ("q", "k", "v", "g")], x["cu"])
    check("o", torch.stack(outs, 1), o_ref.view(B, n + extra, H, D)[:, n:], BF16_TOL)
    check("state", pool[pages.long()], ht_ref, F32_TOL)


# ---- streams, graphs, devices --------------------------------------------------------------------

def test_on_a_stream_of_its_own(gdn):
    x = dev(ref.inputs([150, 70], 2, 2, 128, "bf16", "token", "own", True, seed=25))
    args = [x[n] for n in ("q", "k", "v", "g", "cu")]
    want, wb = gdn.linattn_fwd(*args, x["h0"]), gdn.linattn_bwd(*args, x["dout"], x["h0"], x["dht"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = [a.clone() for a in args]  # on the stream: the call has to follow them there
        got, gb = gdn.linattn_fwd(*late, x["h0"]), gdn.linattn_bwd(*late, x["dout"], x["h0"], x["dht"])
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(gb[n], wb[n]) for n in wb)


def test_two_calls_at_once(gdn):
    """Calls on two streams, each with its own workspace, as each alone (bitwise: nothing is shared)."""
    xs = [dev(ref.inputs([900, 333], 3, 3, 64, "bf16", "token", "own", True, seed=s)) for s in (31, 32)]

    def call(x):
        args = [x[n] for n in ("q", "k", "v", "g", "cu")]
        o, ht = gdn.linattn_fwd(*args, x["h0"], seg_chunks=2)
        return dict(gdn.linattn_bwd(*args, x["dout"], x["h0"], x["dht"], seg_chunks=2), o=o, ht=ht)

    alone = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    both = [[], []]
    for _ in range(5):
        for i, (x, st) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(st):
                both[i].append(call(x))
    torch.cuda.synchronize()
    for i in range(2):
        for got in both[i]:
            assert all(torch.equal(got[n], alone[i][n]) for n in alone[i])


def test_offsets_past_32_bits(gdn):
    """Tensors of more than 2^32 bytes: the last heads' results are those of the last heads alone."""
    T, H, D = 140001, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(33)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, dout = (rnd(T, H, D) for _ in range(4))
    q.mul_(D ** -0.5)
    k.mul_(D ** -0.5)
    g = -0.1 * torch.rand(T, H, generator=gen, device="cuda")
    cu = torch.tensor([0, 100000, T], dtype=torch.int32, device="cuda")
    few = [t[:, -2:].contiguous() for t in (q, k, v, g)]
    o, ht = gdn.linattn_fwd(q, k, v, g, cu, seg_chunks=64)
    of, htf = gdn.linattn_fwd(*few, cu, seg_chunks=64)
    assert ref.rel(o[:, -2:], of) <= 2.0 ** -10 and ref.rel(ht[:, -2:], htf) <= F32_TOL
    assert ref.rel(o[-70:, -1], of[-70:, -1]) <= 2.0 ** -10
    got = gdn.linattn_bwd(q, k, v, g, cu, dout, seg_chunks=64)
    want = gdn.linattn_bwd(*few, cu, dout[:, -2:].contiguous(), seg_chunks=64)
    for n in ("dq", "dk", "dv"):
        assert ref.rel(got[n][:, -2:], want[n]) <= 2.0 ** -10, n
        assert ref.rel(got[n][-70:, -1], want[n][-70:, -1]) <= 2.0 ** -10, n
    assert ref.rel(got["dg"][:, -2:], want["dg"]) <= DG_TOL
    assert ref.rel(got["dh0"][:, -2:], want["dh0"]) <= F32_TOL


def test_graph_replays(gdn):
    """Forward, backward and steps captured into two graphs, replayed on new inputs with eager
    calls between the replays."""
    x = dev(ref.inputs([150, 70], 2, 1, 128, "bf16", "head", "shared", True, seed=26))
    names = ("q", "k", "v", "g", "cu")
    state = torch.randn(2, 2, 128, 128, device="cuda")
    one = {n: x[n][:2].clone() for n in ("q", "k", "v")}

    def passes():
        return gdn.linattn_fwd(*[x[n] for n in names], x["h0"], seg_chunks=1), \
            gdn.linattn_bwd(*[x[n] for n in names], x["dout"], x["h0"], x["dht"], seg_chunks=1)

    def step():
        return gdn.linattn_step(one["q"], one["k"], one["v"], x["g"], state)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        passes(), step()
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        (o, ht), b = passes()
    with torch.cuda.graph(g2):
        so = step()
    for i in range(4):
        for n in ("q", "k", "v", "dout"):
            x[n].copy_(torch.roll(x[n], 1, 0))
        before = state.clone()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        after = state.clone()
        (eo, eh), eb = passes()
        state.copy_(before)
        es = step()
        torch.cuda.synchronize()
        assert torch.equal(o, eo) and torch.equal(ht, eh), i
        assert all(torch.equal(b[n], eb[n]) for n in eb), i
        assert torch.equal(so, es) and torch.equal(after, state), i


def test_debug_mode(gdn):
    """Malformed offsets and pages are errors in debug mode, before and after the launch."""
    x = dev(ref.inputs([64, 64], 2, 2, 64, "bf16", seed=27))
    s = dev(step_inputs(3, 2, 2, 64, "bf16", "token", 28))
    bad = x["cu"].clone()
    bad[1] = 200
    gdn.device_faults(clear=True)
    before = gdn.get_debug()
    gdn.set_debug(True)
    try:
        with pytest.raises(gdn.GdnError):
            gdn.linattn_fwd(x["q"], x["k"], x["v"], x["g"], bad)
        with pytest.raises(gdn.GdnError):
            gdn.linattn_bwd(x["q"], x["k"], x["v"], x["g"], bad, x["dout"])
        gdn.linattn_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"])
        pages = torch.tensor([0, 5, 1], dtype=torch.int32, device="cuda")
        with pytest.raises(gdn.GdnError) as e:
            gdn.linattn_step(s["q"], s["k"], s["v"], s["g"], s["state"], pages)
        assert e.value.status == 9
        gdn.linattn_step(s["q"], s["k"], s["v"], s["g"], s["state"], s["pages"])
        # a page's fault is the fault of the call that named it, not of later forwards
        gdn.set_debug(False)
        gdn.linattn_step(s["q"], s["k"], s["v"], s["g"], s["state"], pages)
        gdn.set_debug(True)
        gdn.linattn_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"])
        beta = torch.full_like(x["g"], 0.5).bfloat16()
        gdn.chunk_fwd(x["q"], x["k"], x["v"], x["g"], beta, x["cu"])
        gdn.set_debug(False)
        gdn.linattn_step(s["q"], s["k"], s["v"], s["g"], s["state"], pages)
        gdn.set_debug(True)
        gdn.pages_free(torch.ones(4, dtype=torch.int32, device="cuda"), s["pages"])
    finally:
        gdn.set_debug(before)
        gdn.device_faults(clear=True)


def test_seeded_mix_of_everything(gdn):
    """Drawn combinations of types, sizes, heads, decays, states, units and document lengths."""
    import random

    rng = random.Random(5)
    for case in range(16):
        dtype, D = rng.choice(["bf16", "f32"]), rng.choice([64, 128])
        H = rng.choice([1, 2, 4])
        Hk = rng.choice([h for h in (1, 2, 4) if H % h == 0])
        lens = [rng.choice([0, 1, 5, 64, rng.randint(1, 200), rng.randint(1, 400)])
                for _ in range(rng.randint(1, 4))] + [3]
        decay, h0 = rng.choice(["token", "head"]), rng.choice(["none", "own", "shared"])
        seg, dht = rng.choice([0, 0, 1, 2, 3]), rng.random() < 0.5
        print(f"[{case}] {dtype} D={D} H={H}/{Hk} {lens} {decay} {h0} dht={dht} seg={seg}", flush=True)
        x = ref.inputs(lens, H, Hk, D, dtype, decay, h0, dht, seed=300 + case)
        run_both(gdn, x, dtype, 0.8, seg_chunks=seg)
