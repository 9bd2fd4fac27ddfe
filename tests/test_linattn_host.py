"""Linear attention and page operators without a GPU: the reference that the GPU tests use, checked
against differences, and what the C ABI and the binding refuse before touching the device."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

import linattn_ref as ref  # noqa: E402


def test_reference_gradients_against_differences():
    """Every gradient of the reference against central differences of its forward."""
    x = ref.inputs([5, 0, 3], 2, 1, 4, "f32", "head", "own", True, seed=1)
    for decay, h0 in (("head", "own"), ("token", "shared")):
        x = ref.inputs([5, 0, 3], 2, 1, 4, "f32", decay, h0, True, seed=1)
        d = {n: t if n == "cu" else t.double() for n, t in x.items()}
        names = ("q", "k", "v", "g")

        def loss(z):
            o, ht = ref.forward(*[z[n] for n in names], z["cu"], z["h0"], 0.7)
            return float((o * d["dout"]).sum() + (ht * d["dht"]).sum())

        got = ref.backward(*[d[n] for n in names], d["cu"], d["dout"], d["h0"], d["dht"], 0.7)
        for n in names + ("h0",):
            num = torch.zeros_like(d[n])
            for i in range(d[n].numel()):
                e = 1e-5
                z = dict(d)
                for s in (1, -1):
                    z[n] = d[n].clone()
                    z[n].view(-1)[i] += s * e
                    num.view(-1)[i] += s * loss(z) / (2 * e)
            assert ref.rel(got["d" + n], num) < 1e-8, n


def test_reference_closed_form():
    """Without decay the state is K^T V; with it each pair is weighed by the decays between."""
    x = ref.inputs([9], 1, 1, 4, "f32", seed=2)
    q, k, v = (x[n].double() for n in ("q", "k", "v"))
    o, ht = ref.forward(q, k, v, torch.zeros(9, 1, dtype=torch.float64), x["cu"])
    assert torch.allclose(ht[0, 0], k[:, 0].T @ v[:, 0])
    g = x["g"].double()
    o, _ = ref.forward(q, k, v, g, x["cu"])
    G = g[:, 0].cumsum(0)
    att = ((q[:, 0] @ k[:, 0].T) * torch.exp(G[:, None] - G[None])).tril()
    assert torch.allclose(o[:, 0], att @ v[:, 0])


@pytest.fixture(scope="module")
def lib():
    from linear_attention_recurrence_prefill_amd import gdn

    if not os.path.exists(gdn.LIB_PATH):
        pytest.fail("libgdn_mi355x.so is not built (run __graft_entry__.build())")
    return gdn.load_library()


FAKE = ctypes.c_void_p(1 << 20)   # aligned, never dereferenced: every call below is refused first
ODD = ctypes.c_void_p((1 << 20) + 4)


def problem(**kw):
    from linear_attention_recurrence_prefill_amd.linattn import LinattnProblem

    p = LinattnProblem(1024, 2, 8, 8, 128, 1, 0, 0, 256, 1.0, 0, 8 * 128 * 128)
    for n, v in kw.items():
        setattr(p, n, v)
    return p


@pytest.mark.parametrize("field,value,status", [
    ("total_tokens", -1, 2), ("total_tokens", 1 << 31, 2), ("num_seqs", 0, 2), ("num_heads", 0, 2),
    ("num_heads", 70000, 2), ("num_k_heads", 3, 2), ("num_k_heads", 16, 2), ("num_k_heads", -1, 2),
    ("head_dim", 96, 2), ("head_dim", 256, 2), ("dtype", 2, 3), ("head_decay", 2, 4),
    ("seg_chunks", -1, 2), ("num_slots", -1, 2), ("scale", float("inf"), 2),
    ("scale", float("nan"), 2), ("reserved", 1, 2), ("h0_seq_stride", -1, 2)])
def test_problem_is_checked(lib, field, value, status):
    p, n = problem(**{field: value}), ctypes.c_size_t(0)
    assert lib.gdn_linattn_fwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == status
    assert lib.gdn_linattn_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == status
    assert lib.gdn_linattn_fwd(ctypes.byref(p), *[FAKE] * 9, 1 << 40, None) == status
    assert lib.gdn_linattn_bwd(ctypes.byref(p), *[FAKE] * 14, 1 << 40, None) == status
    assert lib.gdn_last_error()


def test_too_many_units_are_refused(lib):
    p, n = problem(num_seqs=1 << 25, total_tokens=0), ctypes.c_size_t(0)
    assert lib.gdn_linattn_fwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 2
    p = problem(total_tokens=(1 << 31) - 100, seg_chunks=1)
    assert lib.gdn_linattn_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 2


def test_null_and_misaligned_pointers(lib):
    p = problem()
    for i in range(9):
        args = [FAKE] * 9
        args[i] = None
        if i in (5, 7):  # h0 and ht are optional; workspace is checked on the device's behalf
            continue
        if i == 8:
            continue
        assert lib.gdn_linattn_fwd(ctypes.byref(p), *args, 1 << 40, None) == 1, i
    for i in (0, 1, 2, 5, 6, 7):
        args = [FAKE] * 9
        args[i] = ODD
        assert lib.gdn_linattn_fwd(ctypes.byref(p), *args, 1 << 40, None) == 7, i
    for i in range(12):
        args = [FAKE] * 14
        args[i] = None
        if i in (5, 7):
            continue
        assert lib.gdn_linattn_bwd(ctypes.byref(p), *args, 1 << 40, None) == 1, i
    assert lib.gdn_linattn_fwd_workspace_size(None, None) == 1
    assert lib.gdn_linattn_fwd_workspace_size(ctypes.byref(p), None) == 1


def test_workspace_of_the_split(lib):
    """Unsplit forwards need none; a split one a state per unit and head, its decay, and each
    sequence's first unit."""
    n = ctypes.c_size_t(0)
    size = lambda p, f: (f(ctypes.byref(p), ctypes.byref(n)), n.value)  # noqa: E731
    up = lambda b: (b + 255) // 256 * 256  # noqa: E731
    assert size(problem(num_slots=1), lib.gdn_linattn_fwd_workspace_size) == (0, 0)
    p = problem(seg_chunks=4)  # ceil((16 + 2) / 4) + 2 = 7 units at most
    assert size(p, lib.gdn_linattn_fwd_workspace_size) == \
        (0, up(7 * 8 * 128 * 128 * 4) + up(7 * 8 * 8) + up(8))
    assert size(problem(total_tokens=0), lib.gdn_linattn_bwd_workspace_size) == (0, 0)
    whole = size(problem(num_slots=1), lib.gdn_linattn_bwd_workspace_size)[1]
    assert whole == 3 * up(1024 * 8 * 4) + up(2 * 8 * 4)
    grouped = size(problem(num_slots=1, num_k_heads=2), lib.gdn_linattn_bwd_workspace_size)[1]
    assert grouped - whole == 2 * 1024 * 8 * 128 * 4


@pytest.mark.parametrize("args,status", [
    ((0, 8, 0, 128, 1, 0), 2), ((4, 0, 0, 128, 1, 0), 2), ((1 << 22, 8, 0, 128, 1, 0), 2),
    ((4, 8, 3, 128, 1, 0), 2), ((4, 8, 16, 128, 1, 0), 2), ((4, 8, 0, 96, 1, 0), 2),
    ((4, 8, 0, 128, 3, 0), 3), ((4, 8, 0, 128, 1, 2), 4)])
def test_step_is_checked(lib, args, status):
    assert lib.gdn_linattn_step(*args, 1.0, *[FAKE] * 5, 4, FAKE, FAKE, None) == status


def test_step_pointers(lib):
    ok = (4, 8, 0, 128, 1, 0, 1.0)
    for i in (0, 1, 2, 3, 5, 6):
        a = [FAKE] * 7
        a[i] = None
        assert lib.gdn_linattn_step(*ok, *a[:5], 4, *a[5:], None) == 1, i
    for i in (0, 1, 2, 5, 6):
        a = [FAKE] * 7
        a[i] = ODD
        assert lib.gdn_linattn_step(*ok, *a[:5], 4, *a[5:], None) == 7, i
    assert lib.gdn_linattn_step(*ok, *[FAKE] * 5, 0, FAKE, FAKE, None) == 2
    assert lib.gdn_linattn_step(1 << 16 | 1, 1, *ok[2:], *[FAKE] * 5, 4, FAKE, FAKE, None) == 2
    assert lib.gdn_linattn_step(1 << 22, 2, *ok[2:], *[FAKE] * 4, None, 0, FAKE, FAKE, None) == 2
    assert lib.gdn_linattn_step(4, 8, 0, 128, 1, 0, float("nan"), *[FAKE] * 5, 4, FAKE, FAKE, None) == 2


def test_pages_are_checked(lib):
    n = ctypes.c_size_t(0)
    assert lib.gdn_pages_workspace_size(-1, 0, ctypes.byref(n)) == 2
    assert lib.gdn_pages_workspace_size(4, -1, ctypes.byref(n)) == 2
    assert lib.gdn_pages_workspace_size(4, 4, None) == 1
    assert lib.gdn_pages_workspace_size(100, 50, ctypes.byref(n)) == 0 and n.value >= 4 * 200
    other = ctypes.c_void_p(1 << 30)
    copy = lambda dst=FAKE, P=4, src=other, Ps=4, nb=64, a=FAKE, b=FAKE, n=2, ws=FAKE, wb=1 << 20: \
        lib.gdn_pages_copy(dst, P, src, Ps, nb, a, b, n, ws, wb, None)  # noqa: E731
    assert copy(P=0) == 2 and copy(Ps=0) == 2 and copy(nb=24) == 2 and copy(nb=0) == 2
    assert copy(n=-1) == 2 and copy(dst=None) == 1 and copy(src=None) == 1 and copy(dst=ODD) == 7
    assert copy(a=None) == 1 and copy(b=None) == 1 and copy(ws=None) == 1 and copy(wb=0) == 6
    assert copy(src=ctypes.c_void_p((1 << 20) + 64)) == 2  # the pools overlap but are not the same
    assert copy(n=0) == 0
    fork = lambda pool=FAKE, live=FAKE, P=4, nb=64, par=FAKE, n=2, kids=FAKE, ws=FAKE, wb=1 << 20: \
        lib.gdn_pages_fork(pool, live, P, nb, par, n, kids, ws, wb, None)  # noqa: E731
    assert fork(pool=None) == 1 and fork(live=None) == 1 and fork(par=None) == 1
    assert fork(kids=None) == 1 and fork(P=0) == 2 and fork(nb=8) == 2 and fork(n=-1) == 2
    assert fork(wb=16) == 6 and fork(ws=ODD) == 7 and fork(n=0) == 0
    assert lib.gdn_pages_free(FAKE, 0, FAKE, 1, None) == 2
    assert lib.gdn_pages_free(FAKE, 4, FAKE, -1, None) == 2
    assert lib.gdn_pages_free(None, 4, FAKE, 1, None) == 1
    assert lib.gdn_pages_free(FAKE, 4, FAKE, 0, None) == 0
    comp = lambda pool=FAKE, live=FAKE, P=4, nb=64, remap=FAKE, ws=FAKE, wb=1 << 20: \
        lib.gdn_pages_compact(pool, live, P, nb, remap, ws, wb, None)  # noqa: E731
    assert comp(pool=None) == 1 and comp(live=None) == 1 and comp(remap=None) == 1
    assert comp(P=0) == 2 and comp(nb=40) == 2 and comp(wb=0) == 6
    # lists and flags of one call overlap
    at = lambda i: ctypes.c_void_p((1 << 22) + 4 * i)  # noqa: E731
    assert fork(live=at(0), P=4, par=at(8), kids=at(9), n=2) == 2
    assert fork(live=at(0), P=4, par=at(8), kids=at(3), n=2) == 2
    assert fork(live=at(0), P=4, par=at(3), kids=at(8), n=2) == 2
    assert comp(live=at(0), P=4, remap=at(3)) == 2
    assert lib.gdn_pages_free(at(0), 4, at(3), 2, None) == 2


def test_binding_refuses_bad_tensors():
    """Shapes, types and devices, on CPU tensors: refused before any device call."""
    import linear_attention_recurrence_prefill_amd as gdn

    x = ref.inputs([3, 4], 4, 2, 64, "bf16", seed=3)
    good = dict(q=x["q"], k=x["k"], v=x["v"], g=x["g"], cu_seqlens=x["cu"])
    bad = [dict(q=x["q"][0]), dict(k=x["k"][:5]), dict(v=x["v"][:, :3]), dict(q=x["q"].float()),
           dict(q=x["q"].half(), k=x["k"].half(), v=x["v"].half()), dict(g=x["g"].double()),
           dict(g=x["g"][:, :2]), dict(g=x["g"][0, :3]), dict(cu_seqlens=x["cu"].long()),
           dict(cu_seqlens=x["cu"][:1]), dict(q=x["q"][..., :60], k=x["k"][..., :60])]
    for b in bad + [{}]:  # the last: a CPU tensor is refused too
        with pytest.raises(ValueError):
            gdn.linattn_fwd(**{**good, **b})
        with pytest.raises(ValueError):
            gdn.linattn_bwd(**{**good, **b}, dout=x["dout"])
    state, pages = torch.zeros(9, 4, 64, 64), torch.zeros(7, dtype=torch.int32)
    step = dict(q=x["q"], k=x["k"], v=x["v"], g=x["g"], state=state, pages=pages)
    for b in (dict(state=state.double()), dict(state=state[:, :3]), dict(pages=None),
              dict(pages=pages.long()), dict(pages=pages[:3]), {}):
        with pytest.raises(ValueError):
            gdn.linattn_step(**{**step, **b})
    idx = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: gdn.pages_copy(state, state, idx, idx),
                 lambda: gdn.pages_fork(state, idx, idx), lambda: gdn.pages_free(idx, idx),
                 lambda: gdn.pages_compact(state, idx)):
        with pytest.raises(ValueError):
            call()
