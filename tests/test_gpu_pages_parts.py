"""Copies between a pool and its first pages (gfx950 only; marked ``gpu``): one address, two page counts."""
import random

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_attention_recurrence_prefill_amd as m

    m.load_library()
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def copy_ref(pool, P_dst, P_src, to, frm):
    """(pool after the copy, faults) by the rules of include/gdn_pages.h."""
    want, faults, first = pool.clone(), 0, {}
    ok = [-1 <= t < P_dst and -1 <= f < P_src for t, f in zip(to, frm)]
    for i, t in enumerate(to):
        if ok[i] and t >= 0:
            first.setdefault(t, i)
    for i, (t, f) in enumerate(zip(to, frm)):
        if not ok[i]:
            faults |= 2
        elif t >= 0 and (first[t] != i or (f >= 0 and f != t and f in first)):
            faults |= 4
        elif t >= 0:
            want[t] = pool[f] if f >= 0 else 0
    return want, faults


@pytest.mark.parametrize("P_dst,P_src,n", [(4, 1024, 3), (4, 1024, 300), (1, 2, 1), (700, 64, 90),
                                           (130, 5000, 2500), (64, 64, 40)])
def test_a_pool_and_its_first_pages(gdn, P_dst, P_src, n):
    """Either side the whole pool, the workspace of the stated size between sentinels."""
    rng = random.Random(P_dst + P_src + n)
    pool = torch.randn(max(P_dst, P_src), 8, generator=torch.Generator().manual_seed(n)).cuda()
    low = max(1, P_dst // 2)  # the lower half of dst is written, everything above it read
    to = [rng.randrange(low) if rng.random() < 0.9 else rng.randint(-2, P_dst) for _ in range(n)]
    frm = [rng.randint(min(low, P_src - 1), P_src - 1) if rng.random() < 0.9 else rng.randint(-2, P_src)
           for _ in range(n)]
    to[0], frm[0] = 0, P_src - 1
    want, faults = copy_ref(pool, P_dst, P_src, to, frm)
    need, pad = gdn.gdn_pages_workspace_size(P_dst, n), 1 << 16
    buf = torch.full((need + 2 * pad,), 7, dtype=torch.uint8, device="cuda")
    gdn.device_faults(clear=True)
    gdn.pages_copy(pool[:P_dst], pool[:P_src], ints(to), ints(frm), workspace=buf[pad:pad + need])
    torch.cuda.synchronize()
    assert (buf[:pad] == 7).all() and (buf[pad + need:] == 7).all()
    assert torch.equal(pool, want) and gdn.device_faults(clear=True) == faults
    # the copied pages are copied again from a workspace of the binding's own
    gdn.pages_copy(pool[:P_dst], pool[:P_src], ints([0]), ints([P_src - 1]))
    assert torch.equal(pool[0], pool[P_src - 1]) and gdn.device_faults(clear=True) == 0


def test_parts_that_start_elsewhere_are_refused(gdn):
    pool = torch.zeros(8, 8, device="cuda")
    with pytest.raises(gdn.GdnError, match="overlap"):
        gdn.pages_copy(pool[1:], pool, ints([0]), ints([5]))
    with pytest.raises(gdn.GdnError, match="overlap"):
        gdn.pages_copy(pool, pool[2:4], ints([0]), ints([1]))
    gdn.pages_copy(pool[:4], pool[4:], ints([0]), ints([1]))  # apart: two pools
