"""Linear attention beyond the first rounds of its loops, against the definition in 64 bits
(tests/linattn_ref.py; gfx950 only; marked ``gpu``): more units of a sequence than the scan holds ahead
(16) and than one batch of decays (64), units of more chunks than one block of dg's scan (64), more
sequences than one wave (64), than are ranked by length (256) and than dg's sum over units takes at
once (256), and a step's rows beyond the first 256.

Every result is judged for each (document, head) and, in bf16, each block of 64 rows, so that one wrong
row fails.  Tolerances, relative L2:
  bf16 outputs: one rounding of at most 2^-8 of each value, plus 2^-16 of the terms of a sum that is
    itself rarely below a sixteenth of them: 2^-8 + 2^-12 in any block.  Over 4096 values and more the
    roundings' mean square counts, at most (2^-8)^2 / 3, whose own deviation over n values is below
    sqrt(0.8 / n) of it, 1.4 % at 4096: 2^-8 / sqrt 3 + 2^-12.
  fp32 results (ht, dh0): an element passes through at most some 10^3 roundings of 2^-24 whose errors
    are independent, sqrt(10^3) 2^-24 = 2e-6; twice that.
  dg is a difference of sums over its unit and is held to what it is summed from, not to itself: each
    q_s . dq_s and k_s . dk_s is off by at most the same 4e-6 of |q_s| |dq_s| and |k_s| |dk_s|,
    independently, so dg_t by 4e-6 of the root of their summed squares over the document (the pairs
    within a chunk are terms of the same products)."""
import pytest

torch = pytest.importorskip("torch")

import linattn_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BLOCK_TOL, BF16_TOL, F32_TOL = 2.0 ** -8 + 2.0 ** -12, 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -12, 4e-6


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_attention_recurrence_prefill_amd as m

    m.load_library()
    return m


def rel(x, want):
    x, want = x.double().cpu(), want.double().cpu()
    den = float(want.norm())
    return float((x - want).norm()) / (den if den > 0 else 1.0)


def check_rows(name, got, want, cu, bf16):
    """got, want [T, heads, D], by document, head and block of rows."""
    assert torch.isfinite(got.float()).all(), name
    worst = 0.0
    for n in range(len(cu) - 1):
        t0, t1 = int(cu[n]), int(cu[n + 1])
        for h in range(want.shape[1]):
            parts = [(t0, t1)]
            if bf16:
                parts += [(b, min(b + 64, t1)) for b in range(t0, t1, 64)]
            for a, b in parts:
                if a == b:
                    continue
                x, w = got[a:b, h], want[a:b, h]
                tol = F32_TOL if not bf16 else BF16_TOL if w.numel() >= 4096 else BLOCK_TOL
                err = rel(x, w)
                worst = max(worst, err / tol)
                assert err <= tol, f"{name}: document {n}, head {h}, rows {a}..{b}: {err:.3e} > {tol:.1e}"
    print(f"  {name}: worst {worst:.2f} of its tolerance", flush=True)


def check_states(name, got, want):
    for h in range(want.shape[-3]):
        for n in range(want.shape[0]):
            err = rel(got[n, h], want[n, h])
            assert err <= F32_TOL, f"{name}: {n}, head {h}: {err:.3e}"


def check_dg(got, want, cu, rows):
    """rows: per token and head |q| |dq| and |k| |dk|, squared and summed.  A decay per head takes the
    sum over t, to which token s brings its error as often as there are tokens t before it."""
    got, want, worst = got.double().cpu(), want.double(), 0.0
    docs = [(int(cu[n]), int(cu[n + 1])) for n in range(len(cu) - 1) if cu[n] < cu[n + 1]]
    if got.dim() == 1:
        often = torch.cat([torch.arange(1, b - a + 1) for a, b in docs]).double()[:, None]
        bound = F32_TOL * (rows * often ** 2).sum(0).sqrt()
        worst = float(((got - want).abs() / bound).max())
    for a, b in docs if got.dim() == 2 else []:
        bound = F32_TOL * rows[a:b].sum(0).sqrt()
        worst = max(worst, float(((got[a:b] - want[a:b]).abs().amax(0) / bound).max()))
    print(f"  dg: worst {worst:.2f} of its tolerance", flush=True)
    assert worst <= 1


def run(gdn, x, dtype, seg, fwd=True, bwd=True):
    d = {n: None if t is None else (t.float() if n in ("h0", "dht") else t).cuda() for n, t in x.items()}
    r = {n: t if t is None or n == "cu" else t.float().double() for n, t in x.items()}
    args, rargs = ([z[n] for n in ("q", "k", "v", "g", "cu")] for z in (d, r))
    cu, bf16 = x["cu"], dtype == "bf16"
    if fwd:
        o, ht = gdn.linattn_fwd(*args, d["h0"], scale=0.7, seg_chunks=seg)
        o_ref, ht_ref = ref.forward(*rargs, r["h0"], 0.7)
        check_rows("o", o, o_ref, cu, bf16)
        check_states("ht", ht, ht_ref)
    if bwd:
        got = gdn.linattn_bwd(*args, d["dout"], d["h0"], d["dht"], scale=0.7, seg_chunks=seg)
        want = ref.backward(*rargs, r["dout"], r["h0"], r["dht"], 0.7)
        for n in ("dq", "dk", "dv"):
            check_rows(n, got[n], want[n], cu, bf16)
        check_states("dh0", got["dh0"] if got["dh0"].dim() == 4 else got["dh0"][None],
                     want["dh0"] if want["dh0"].dim() == 4 else want["dh0"][None])
        H, Hk = r["v"].shape[1], r["q"].shape[1]
        norm = lambda a: a.norm(dim=-1).repeat_interleave(H // Hk, dim=1)  # noqa: E731
        rows = (norm(r["q"]) * norm(want["dq"])) ** 2 + (norm(r["k"]) * norm(want["dk"])) ** 2
        check_dg(got["dg"], want["dg"], cu, rows)


@pytest.mark.parametrize("dtype,D,H,Hk", [("bf16", 64, 2, 1), ("bf16", 128, 1, 1), ("f32", 64, 1, 1)])
@pytest.mark.parametrize("seg", [1, 3, 1000])
def test_many_units_and_long_units(gdn, dtype, D, H, Hk, seg):
    """4301 tokens: 68 units of one chunk, 23 of three, or one unit of 68 chunks."""
    x = ref.inputs([4301, 70], H, Hk, D, dtype, "token", "own", True, seed=51)
    run(gdn, x, dtype, seg)


@pytest.mark.parametrize("seg", [1, 1000])
def test_long_units_with_a_decay_per_head(gdn, seg):
    x = ref.inputs([130, 4301], 2, 2, 64, "bf16", "head", "none", False, seed=52, g_mu=-4.0)
    run(gdn, x, "bf16", seg)


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("N", [70, 256, 300])
@pytest.mark.parametrize("seg", [0, 1])
def test_many_documents(gdn, decay, N, seg):
    """Ragged documents, some empty, whole (longest first up to 256 of them) and in units."""
    gen = torch.Generator().manual_seed(53 + N)
    lens = torch.randint(0, 30, (N,), generator=gen).tolist()
    for i in range(0, N, 9):  # more chunks than their neighbours, in every group of 64
        lens[i] = 60 + 7 * (i % 23)
    lens[N // 2], lens[-1] = 0, 77
    x = ref.inputs(lens, 2, 1, 64, "bf16", decay, "shared" if seg else "own", True, seed=54)
    run(gdn, x, "bf16", seg)


def test_many_heads_row_by_row(gdn):
    """More workgroups than CUs, every block of rows of every head."""
    x = ref.inputs([450, 70], 2, 2, 128, "bf16", "token", "own", True, seed=55)
    r = {n: t if n == "cu" else t.float().double() for n, t in x.items()}
    o_ref, _ = ref.forward(*[r[n] for n in ("q", "k", "v", "g", "cu")], r["h0"])
    want = ref.backward(*[r[n] for n in ("q", "k", "v", "g", "cu")], r["dout"], r["h0"], r["dht"])
    want["o"] = o_ref
    many = lambda t: t.repeat(*(140 if i == 1 else 1 for i in range(t.dim())))  # noqa: E731
    d = {n: (t if n == "cu" else many(t.float() if n in ("h0", "dht") else t)).cuda() for n, t in x.items()}
    args = [d[n] for n in ("q", "k", "v", "g", "cu")]
    for seg in (0, 2, 1000):
        got = gdn.linattn_bwd(*args, d["dout"], d["h0"], d["dht"], seg_chunks=seg)
        got["o"] = gdn.linattn_fwd(*args, d["h0"], seg_chunks=seg)[0]
        for n in ("o", "dq", "dk", "dv"):
            w = want[n].cuda()
            for a in list(range(0, 450, 64)) + [450, 514]:
                b = min(a + 64, 450) if a < 450 else min(a + 64, 520)
                e = (got[n][a:b].double().view(b - a, 140, 2, 128) - w[a:b, None]).norm(dim=(0, 3))
                err = float((e / w[a:b].norm(dim=(0, 2))).max())
                assert err <= BLOCK_TOL, f"{n}, seg {seg}, rows {a}..{b}: {err:.3e}"


def test_step_of_many_rows(gdn):
    """300 rows on pages, with pages that a row more than 256 rows earlier has, and rows without one."""
    B, H, D, P = 300, 2, 64, 320
    x = ref.inputs([1] * B, H, 1, D, "bf16", "token", seed=56)
    gen = torch.Generator().manual_seed(57)
    state = torch.randn(P, H, D, D, generator=gen)
    pages = torch.randperm(P, generator=gen)[:B].to(torch.int32)
    pages[270], pages[299], pages[280], pages[290] = pages[3], pages[42], -1, pages[289]
    zero = [270, 280, 290, 299]
    rows = torch.tensor([b for b in range(B) if b not in zero])
    pool = state.cuda()
    gdn.device_faults(clear=True)
    o = gdn.linattn_step(*(x[n].cuda() for n in ("q", "k", "v", "g")), pool, pages.cuda())
    assert gdn.device_faults(clear=True) == 4
    q, k = (x[n].double().repeat_interleave(H, dim=1)[rows] for n in ("q", "k"))
    v, g = x["v"].double()[rows], x["g"].double()[rows]
    S = g.exp()[..., None, None] * state.double()[pages.long()[rows]] + \
        k[..., :, None] * v[..., None, :]
    want = (q[..., :, None] * S).sum(-2)
    for i, b in enumerate(rows.tolist()):
        assert rel(o[b], want[i]) <= BLOCK_TOL and rel(pool[pages[b]], S[i]) <= F32_TOL, b
    assert (o[zero] == 0).all()
    rest = torch.ones(P, dtype=torch.bool)
    rest[pages.long()[rows]] = False
    assert torch.equal(pool.cpu()[rest], state[rest])
