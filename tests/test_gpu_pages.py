"""The operators on a pool's pages against plain indexing on the host (gfx950 only; marked ``gpu``).
Pages are moved, not computed: every comparison is exact."""
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


def pool_of(P, shape, dtype=torch.float32, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(P, *shape, generator=gen).to(dtype).cuda()


# page sizes: one 16-byte unit, a ragged piece of 16 KiB, several pieces, a state of two heads
SHAPES = [((4,), torch.float32), ((1028,), torch.float32), ((9, 1000), torch.bfloat16),
          ((2, 64, 64), torch.float32)]


@pytest.mark.parametrize("shape,dtype", SHAPES)
def test_copy_between_pools(gdn, shape, dtype):
    src, dst = pool_of(5, shape, dtype, 1), pool_of(7, shape, dtype, 2)
    want = dst.clone()
    to, frm = [6, 0, -1, 3, 2], [0, 4, 1, -1, 4]
    for t, f in zip(to, frm):
        if t >= 0:
            want[t] = src[f] if f >= 0 else 0
    out = gdn.pages_copy(dst, src, ints(to), ints(frm))
    torch.cuda.synchronize()
    assert out is dst and torch.equal(dst, want)
    gdn.pages_copy(dst, src, ints([]), ints([]))
    assert torch.equal(dst, want)


def test_copy_refuses_pairs_that_race(gdn):
    """In one pool: a destination named twice keeps its first pair, a pair whose source another pair
    overwrites is left out, a page onto itself is nothing; pages outside the pools are left out."""
    pool = pool_of(8, (64,), seed=3)
    gdn.device_faults(clear=True)
    want = pool.clone()
    want[1] = pool[0]
    gdn.pages_copy(pool, pool, ints([1, 1, 2, 5]), ints([0, 3, 1, 5]))
    assert torch.equal(pool, want) and gdn.device_faults(clear=True) == 4
    gdn.pages_copy(pool, pool, ints([8, -2, 3]), ints([0, 0, 9]))
    assert torch.equal(pool, want) and gdn.device_faults(clear=True) == 2
    dst = pool_of(4, (64,), seed=4)
    keep = dst.clone()
    keep[0] = pool[7]
    gdn.pages_copy(dst, pool, ints([0, 0]), ints([7, 6]))
    assert torch.equal(dst, keep) and gdn.device_faults(clear=True) == 4


@pytest.mark.parametrize("same", [True, False])
def test_copy_of_long_lists(gdn, same):
    """Lists beyond one round of the checking workgroup, with pages named often and bad pages."""
    rng = random.Random(11)
    P, n = 700, 2500
    src = pool_of(P, (8,), seed=12)
    dst = src if same else pool_of(P, (8,), seed=13)
    to = [rng.choice([-1, P, rng.randrange(P)]) for _ in range(n)]
    frm = [rng.choice([-1, rng.randrange(P), rng.randrange(-2, P + 1)]) for _ in range(n)]
    if same:  # half of the pages are sources only
        to = [t - t % 2 if 0 <= t < P else t for t in to]
        frm = [f if rng.random() < 0.1 or not 0 <= f < P else f | 1 for f in frm]
    ok = [-1 <= t < P and -1 <= f < P for t, f in zip(to, frm)]
    written, want, faults = {}, dst.clone(), 0
    for i, t in enumerate(to):
        if ok[i] and t >= 0:
            written.setdefault(t, i)
    for i, (t, f) in enumerate(zip(to, frm)):
        if not ok[i]:
            faults |= 2
        elif t >= 0 and (written[t] != i or (same and f >= 0 and f != t and f in written)):
            faults |= 4
        elif t >= 0:
            want[t] = src[f] if f >= 0 else 0
    gdn.device_faults(clear=True)
    gdn.pages_copy(dst, src, ints(to), ints(frm))
    assert torch.equal(dst, want) and gdn.device_faults(clear=True) == faults


def fork_ref(pool, live, parents):
    pool, live, children = pool.clone(), list(live), []
    free = [p for p, x in enumerate(live) if not x]
    took = []
    for p in parents:
        ok = p == -1 or (0 <= p < len(live) and live[p])
        c = free.pop(0) if ok and free else -1
        children.append(c)
        if c >= 0:
            took.append((c, p))
    for c, p in took:
        pool[c] = pool[p] if p >= 0 else 0
        live[c] = 1
    return pool, live, children


@pytest.mark.parametrize("P,n,seed", [(1, 1, 0), (6, 3, 1), (40, 25, 2), (40, 60, 3), (2500, 1300, 4),
                                      (1024, 1024, 5), (1024, 1025, 6), (1025, 30, 7)])
def test_fork(gdn, P, n, seed):
    """Fewer and more parents than free pages, the same parent many times, new (zero) pages, parents
    that are not live; a pool beyond one round of the planning workgroup."""
    rng = random.Random(seed)
    live = [rng.choice([0, 1, 5]) for _ in range(P)]
    parents = [rng.choice([-1, rng.randrange(P), rng.randrange(P)]) for _ in range(n)]
    pool = pool_of(P, (8,), seed=seed)
    want, live_ref, kids = fork_ref(pool, live, parents)
    lv = ints(live)
    gdn.device_faults(clear=True)
    got = gdn.pages_fork(pool, lv, ints(parents))
    torch.cuda.synchronize()
    assert got.tolist() == kids
    assert torch.equal(pool, want)
    assert [x != 0 for x in lv.tolist()] == [x != 0 for x in live_ref]
    bad = 2 if any(p >= 0 and not live[p] for p in parents) else 0
    full = 8 if sum(p == -1 or live[p] != 0 for p in parents) > sum(not x for x in live) else 0
    assert gdn.device_faults(clear=True) == bad | full


def test_fork_into_a_given_list(gdn):
    pool, lv, kids = pool_of(4, (8,)), ints([1, 0, 1, 0]), ints([9, 9, 9])
    assert gdn.pages_fork(pool, lv, ints([2, 0, 0]), children=kids) is kids
    assert kids.tolist() == [1, 3, -1] and lv.tolist() == [1, 1, 1, 1]
    assert torch.equal(pool[1], pool[2]) and torch.equal(pool[3], pool[0])
    assert gdn.device_faults(clear=True) == 8
    for bad in (kids, kids[:2]):  # the list itself, and a part of it
        with pytest.raises(RuntimeError, match="overlap"):
            gdn.pages_fork(pool, lv, kids[1:] if bad is not kids else kids, children=bad)
    with pytest.raises(RuntimeError, match="overlap"):
        gdn.pages_free(lv, lv[1:])


def test_fork_of_pages_outside_the_pool(gdn):
    pool, lv = pool_of(4, (8,)), ints([1, 0, 0, 0])
    before = pool.clone()
    gdn.device_faults(clear=True)
    kids = gdn.pages_fork(pool, lv, ints([4, -2, 0, 1 << 30]))
    assert kids.tolist() == [-1, -1, 1, -1] and lv.tolist() == [1, 1, 0, 0]
    before[1] = before[0]
    assert torch.equal(pool, before) and gdn.device_faults(clear=True) == 2


def test_free(gdn):
    lv = ints([1] * 3000)
    gdn.device_faults(clear=True)
    gdn.pages_free(lv, ints([0, 7, 7, -1, 2999]))
    gdn.pages_free(lv, ints([7] * 1000))
    gdn.pages_free(lv, ints([]))
    want = [0 if p in (0, 7, 2999) else 1 for p in range(3000)]
    assert lv.tolist() == want and gdn.device_faults() == 0
    gdn.pages_free(lv, ints([3000, -5, 1]))
    want[1] = 0
    assert lv.tolist() == want and gdn.device_faults(clear=True) == 2


@pytest.mark.parametrize("P,share,shape,dtype", [
    (1, 0.0, (4,), torch.float32), (1, 1.0, (4,), torch.float32), (2, 0.5, (4,), torch.float32),
    (33, 0.4, (1028,), torch.float32), (64, 0.0, (8,), torch.float32),
    (64, 1.0, (8,), torch.float32), (65, 0.6, (9, 1000), torch.bfloat16),
    (2600, 0.5, (8,), torch.float32), (1024, 0.5, (8,), torch.float32),
    (1024, 1.0, (8,), torch.float32), (1024, 0.0, (8,), torch.float32), (1025, 0.7, (8,), torch.float32)])
def test_compact(gdn, P, share, shape, dtype):
    rng = random.Random(P)
    live = [int(rng.random() < share) for _ in range(P)]
    pool, lv = pool_of(P, shape, dtype, 5), ints([3 * x for x in live])
    before = pool.clone()
    remap = gdn.pages_compact(pool, lv)
    torch.cuda.synchronize()
    n = sum(live)
    holes = [p for p in range(n) if not live[p]]
    want = [(p if p < n else holes.pop(0)) if live[p] else -1 for p in range(P)]
    assert remap.tolist() == want
    assert lv.tolist() == [1] * n + [0] * (P - n)
    for p in range(P):
        if live[p]:
            assert torch.equal(pool[want[p]], before[p]), p
    assert torch.equal(pool[n:], before[n:])


def test_a_serving_run(gdn):
    """Prompts, their states in a pool, forks, steps, sequences that end, compaction and steps again
    on the compacted batch, against a dict of states kept on the host in 64 bits."""
    H, D, P = 2, 64, 12
    gen = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    g = -torch.rand(H, generator=gen)
    pool = torch.zeros(P, H, D, D, device="cuda")
    live = torch.zeros(P, dtype=torch.int32, device="cuda")
    q, k, v = (rnd(90, H, D) / 8 for _ in range(3))
    cu = ints([0, 40, 90])
    _, ht = gdn.linattn_fwd(q.cuda(), k.cuda(), v.cuda(), g.cuda(), cu)
    first = gdn.pages_fork(pool, live, ints([-1, -1]))
    gdn.pages_copy(pool, ht, first, ints([0, 1]))
    import linattn_ref as ref

    _, S = ref.forward(q.double(), k.double(), v.double(), g.double(), cu.cpu())
    states = {0: S[0], 1: S[1]}  # by page
    kids = gdn.pages_fork(pool, live, ints([1, 0, 1, 1]))
    assert kids.tolist() == [2, 3, 4, 5]
    states.update({2: S[1], 3: S[0], 4: S[1], 5: S[1]})

    def steps(pages):
        for _ in range(3):
            q, k, v = (rnd(len(pages), H, D) / 8 for _ in range(3))
            o = gdn.linattn_step(q.cuda(), k.cuda(), v.cuda(), g.cuda(), pool, ints(pages))
            for i, p in enumerate(pages):
                if p < 0:
                    continue
                states[p] = g.double().exp()[:, None, None] * states[p] + \
                    k[i].double()[:, :, None] * v[i].double()[:, None, :]
                want = (q[i].double()[:, :, None] * states[p]).sum(1)
                assert ref.rel(o[i], want) <= 4e-6

    steps([0, 1, 2, 3, 4, 5, -1])
    gdn.pages_free(live, ints([0, 3]))
    remap = gdn.pages_compact(pool, live).tolist()
    assert remap[:6] == [-1, 1, 2, -1, 0, 3]
    states = {remap[p]: s for p, s in states.items() if remap[p] >= 0}
    steps([0, 1, 2, 3])
    for p, s in states.items():
        assert ref.rel(pool[p], s) <= 4e-6
    assert gdn.device_faults() == 0


def test_graph_replays(gdn):
    """Free, compact and fork captured once and replayed: every replay does what the eager calls do."""
    P, n = 20, 6
    pool, live = pool_of(P, (2, 64, 64), seed=9), ints([1] * P)
    gone, parents = ints([3, 19, 7, 8, 11, 2]), ints([0] * n)

    def turn(pool, live):
        gdn.pages_free(live, gone)
        remap = gdn.pages_compact(pool, live)
        return remap, gdn.pages_fork(pool, live, parents)

    p2, l2 = pool.clone(), live.clone()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        turn(p2.clone(), l2.clone())
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        remap, kids = turn(pool, live)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        r2, k2 = turn(p2, l2)
        torch.cuda.synchronize()
        assert torch.equal(remap, r2) and torch.equal(kids, k2)
        assert torch.equal(pool, p2) and torch.equal(live, l2)


def test_pages_past_32_bits(gdn):
    """A pool of more than 2^32 bytes: offsets of its last pages are 64-bit."""
    P, n = 5, 1 << 28  # five pages of 1 GiB
    pool = torch.empty(P, n, device="cuda")
    for p in range(P):
        pool[p].fill_(p)
    live = ints([0, 1, 0, 0, 1])
    remap = gdn.pages_compact(pool, live)
    assert remap.tolist() == [-1, 1, -1, -1, 0]
    assert (pool[0] == 4).all() and (pool[1] == 1).all() and (pool[4] == 4).all()
    gdn.pages_copy(pool, pool, ints([4]), ints([1]))
    assert (pool[4] == 1).all()
