"""Linear attention where its sums cancel (gfx950 only; marked ``gpu``): keys with a common direction
and queries nearly orthogonal to it, so that S^T q is far smaller than the state's elements allow, and
the mirrored case for dv.  Against the definition in 64 bits (tests/linattn_ref.py).

Tolerance.  A bf16 output is rounded once, by at most 2^-8 of itself, rho = 2^-8 / sqrt 3 in the mean
square.  Operands that are not inputs are sums of two bf16 terms, so each is off by at most 2^-16 of
itself, 2^-16 / sqrt 3 in the mean square: the state's elements S_ij, of which o_j takes q_i S_ij; the
pairs' weights w_t = D_t (q . k_t), of which o_j takes w_t v_tj; and the decayed v_tj that enter the
state, of which o_j takes the same w_t v_tj.  These errors are independent from element to element, so
that of o_j is at most 2^-16 / sqrt 3 times the root of the summed squares of those three sets of
terms, whatever their sum.  fp32's own rounding (2^-24) is far below."""
import pytest

torch = pytest.importorskip("torch")

import linattn_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
RHO, TWO_TERMS = 2.0 ** -8 / 3 ** 0.5, 2.0 ** -16 / 3 ** 0.5


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_attention_recurrence_prefill_amd as m

    m.load_library()
    return m


def cancelling(lens, H, D, weight, seed):
    """x (queries) orthogonal to the direction that y (keys) share with `weight` against unit noise, z
    (values) of mean one, slow decays; bf16, on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    T = sum(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    u = unit(rand(H, D))
    x = rand(T, H, D)
    x = unit(x - (x * u).sum(-1, keepdim=True) * u).bfloat16()
    y = unit(weight * u + unit(rand(T, H, D))).bfloat16()
    z = (1 + rand(T, H, D)).bfloat16()
    g = (-0.002 * (1 + 0.5 * torch.rand(T, H, generator=gen, dtype=torch.float64))).float()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return x, y, z, g, torch.tensor(cu, dtype=torch.int32)


def spread(x, y, z, g, lens, rev):
    """Root of the summed squares of the terms that x's outputs are summed from (see the file's head);
    rev: the recurrence runs backward in time."""
    out, t0 = torch.empty_like(z), 0
    for n in lens:
        xs, ys, zs, gs = (a[t0:t0 + n].permute(1, 0, *range(2, a.dim())) for a in (x, y, z, g))
        G = gs.cumsum(1)
        diff = G[:, :, None] - G[:, None, :]
        diff = -diff if rev else diff
        keep = torch.ones(n, n, dtype=torch.bool)
        keep = keep.triu() if rev else keep.tril()
        D = diff.masked_fill(~keep, float("-inf")).exp()
        pairs = (D * (xs @ ys.transpose(1, 2))) ** 2 @ zs ** 2
        S = torch.zeros(xs.shape[0], xs.shape[2], zs.shape[2], dtype=torch.float64)
        state = torch.empty_like(zs)
        for i in range(n):
            t = n - 1 - i if rev else i
            # forward: decayed by token t, then t's own term; backward: by token t + 1
            at = t + 1 if rev else t
            if 0 < i:
                S = gs[:, at].exp()[:, None, None] * S
            S = S + ys[:, t, :, None] * zs[:, t, None, :]
            state[:, t] = ((xs[:, t, :, None] * S) ** 2).sum(1)
        out[t0:t0 + n] = (state + 2 * pairs).sqrt().transpose(0, 1)
        t0 += n
    return out


def check(name, got, want, terms):
    """Per head: one rounding of the output and the two-term roundings of what it is summed from."""
    for h in range(want.shape[1]):
        w, d = want[:, h].norm(), (got[:, h].double().cpu() - want[:, h]).norm()
        tol = RHO + TWO_TERMS * float(terms[:, h].norm() / w)
        err = float(d / w)
        print(f"  {name}[{h}]: {err:.2e} (tol {tol:.2e})", flush=True)
        assert err <= tol, f"{name}[{h}]: {err:.3e} > {tol:.2e}"


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("weight", [0.0, 1.0, 4.0])
@pytest.mark.parametrize("seg", [3, 5, 1000])
def test_outputs_of_correlated_keys(gdn, D, weight, seg):
    lens = [1024, 333]
    x, y, z, g, cu = cancelling(lens, 2, D, weight, 41)
    want, _ = ref.forward(x.double(), y.double(), z.double(), g.double(), cu)
    terms = spread(x.double(), y.double(), z.double(), g.double(), lens, False)
    got, _ = gdn.linattn_fwd(*(t.cuda() for t in (x, y, z, g, cu)), seg_chunks=seg)
    check("o", got, want, terms)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("weight", [0.0, 1.0, 4.0])
@pytest.mark.parametrize("seg", [3, 5, 1000])
def test_value_gradients_of_correlated_queries(gdn, D, weight, seg):
    """dv_i = sum_{t >= i} D (q_t . k_i) do_t: queries with a common direction, keys orthogonal to it."""
    lens = [1024, 333]
    k, q, dout, g, cu = cancelling(lens, 2, D, weight, 42)
    v = torch.ones_like(dout)
    want = ref.backward(q.double(), k.double(), v.double(), g.double(), cu, dout.double())["dv"]
    terms = spread(k.double(), q.double(), dout.double(), g.double(), lens, True)
    got = gdn.linattn_bwd(*(t.cuda() for t in (q, k, v, g, cu, dout)), seg_chunks=seg)["dv"]
    check("dv", got, want, terms)


def test_a_sequence_alone_and_in_a_batch(gdn):
    """One sequence whole, in units of every kind, and in a batch whose size changes the units that the
    library chooses: the same numbers but for roundings that a last bit tips.  The sums differ by at
    most e = 2^-16 of the terms, a few times the outputs' size on these rows; a rounding of steps 2^-7
    is tipped with probability e / 2^-7 and then moves its value by 2^-7 at most: 2^-10 in the mean
    square holds for e up to 2^-13."""
    T, H, D = 900, 2, 128
    x = ref.inputs([T], H, H, D, "bf16", "token", "own", False, seed=43)
    d = {n: None if t is None else (t.float() if n == "h0" else t).cuda() for n, t in x.items()}
    args = [d[n] for n in ("q", "k", "v", "g", "cu")]
    o, _ = gdn.linattn_fwd(*args, d["h0"])
    dv = gdn.linattn_bwd(*args, d["dout"], d["h0"])["dv"]
    for seg in (1, 4, 5, 15):
        o2, _ = gdn.linattn_fwd(*args, d["h0"], seg_chunks=seg)
        dv2 = gdn.linattn_bwd(*args, d["dout"], d["h0"], seg_chunks=seg)["dv"]
        assert ref.rel(o2, o) <= 2.0 ** -10 and ref.rel(dv2, dv) <= 2.0 ** -10, seg
    for others in (7, 600):
        more = lambda t: torch.cat([t] + [t] * others)  # noqa: E731
        cu = torch.arange(0, T * (others + 1) + 1, T, dtype=torch.int32, device="cuda")
        batch = [more(t) for t in args[:4]] + [cu]
        o2, _ = gdn.linattn_fwd(*batch, more(d["h0"]))
        dv2 = gdn.linattn_bwd(*batch, more(d["dout"]), more(d["h0"]))["dv"]
        assert ref.rel(o2[:T], o) <= 2.0 ** -10 and ref.rel(dv2[:T], dv) <= 2.0 ** -10, others
        assert ref.rel(o2[-T:], o) <= 2.0 ** -10 and ref.rel(dv2[-T:], dv) <= 2.0 ** -10, others
