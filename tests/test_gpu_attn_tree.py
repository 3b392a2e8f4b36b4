"""Tree attention over a paged cache against the plain fp64 form."""
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def api():
    from gated_delta_rule_132_b200 import attn
    return attn


def cache(seed, ctx, n_draft, page, Hq, Hkv, d, dtype, spare=2, M=None):
    """Random pools with shuffled pages, and q for n_draft tokens per sequence."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = len(ctx)
    need = [-(-(c + n_draft) // page) for c in ctx]
    P = sum(need) + spare
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    M = max(max(need), 1) if M is None else M
    table = torch.full((N, M), -1, dtype=torch.int32, device="cuda")
    a = 0
    for n, c in enumerate(need):
        table[n, :c] = perm[a:a + c]
        a += c
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    return (mk(N, n_draft, Hq, d), mk(P, Hkv, page, d), mk(P, Hkv, page, d), table,
            torch.tensor(ctx, dtype=torch.int32, device="cuda"))


def random_parents(seed, N, n_draft, lost=0.0):
    g = torch.Generator().manual_seed(seed)
    p = torch.empty(N, n_draft, dtype=torch.int32)
    for i in range(n_draft):
        p[:, i] = torch.randint(-1, max(i, 0), (N,), generator=g) if i else -1
    if lost:
        odd = torch.rand(N, n_draft, generator=g) < lost
        p = torch.where(odd, torch.randint(-9, -1, p.shape, generator=g).int(), p)
    return p.cuda()


def check(x, parents, scale=None):
    q, kp, vp, table, ctx = x
    s = q.shape[-1] ** -0.5 if scale is None else scale
    o, lse = api().kda_attn_tree(q, kp, vp, table, ctx, parents=parents, scale=scale)
    ro, rl, to, tl = R.attn_tree(q, kp, vp, table, ctx, parents, s)
    R.close(o, ro, to)
    R.close(lse, rl, tl)
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("page", [1, 16, 64, 1024])
def test_single_tokens(page, d, dtype):
    check(cache(1, [0, 1, 15, 16, 17, 63, 64, 65, 200, 1029], 1, page, 4, 2, d, DT[dtype]), None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n_draft", [2, 3, 7, 8, 9, 16, 31, 33, 64])
def test_trees(n_draft, dtype):
    x = cache(n_draft, [0, 5, 64, 130, 700], n_draft, 16, 8, 2, 128, DT[dtype])
    check(x, random_parents(n_draft, 5, n_draft))
    check(x, None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (3, 1, 128), (6, 3, 32), (8, 8, 64), (5, 1, 128), (16, 2, 64),
                                      (32, 1, 128), (40, 2, 32)])
def test_heads(Hq, Hkv, d, dtype):
    x = cache(3, [0, 77, 300], 5, 32, Hq, Hkv, d, DT[dtype])
    check(x, random_parents(4, 3, 5))
    x = cache(3, [0, 77, 300], 1, 32, Hq, Hkv, d, DT[dtype])
    check(x, None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_absent_tokens(dtype):
    """Parents that are no earlier draft, forward and self references, and what hangs from them."""
    x = cache(5, [0, 40, 129, 7], 12, 16, 4, 2, 64, DT[dtype])
    o, lse = check(x, random_parents(6, 4, 12, lost=0.4))
    bad = torch.tensor([[-2] * 12, [-1, 1, 0, 2, 9, 3, -1, 100, 7, 6, 2 ** 31 - 1, -2 ** 31],
                        [-1] + [0] * 11, list(range(-1, 11))], dtype=torch.int32, device="cuda")
    o, lse = check(x, bad)
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_masked_places_do_not_matter(bad, dtype):
    """Drafts off a token's path, the rest of its last page and unused pages may hold anything."""
    ctx, n_draft, page = [3, 60, 200], 6, 16
    q, kp, vp, table, c = cache(7, ctx, n_draft, page, 4, 2, 64, DT[dtype])
    parents = torch.tensor([[-1, -1, 0, 0, 1, 2]] * 3, dtype=torch.int32, device="cuda")
    o, lse = check((q, kp, vp, table, c), parents)
    used = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
    for n, x in enumerate(ctx):
        for t in range(x + n_draft):
            used[table[n, t // page].long(), t % page] = True
        used[table[n, (x + 1) // page].long(), (x + 1) % page] = False  # draft 1: ancestor of draft 4 only
    kp, vp = (torch.where(used[:, None, :, None], x, bad) for x in (kp, vp))
    o2, lse2 = api().kda_attn_tree(q, kp, vp, table, c, parents=parents)
    keep = [0, 2, 3, 5]
    # The exact result is the same, so both runs are within its bound; they need not be the
    # same bits, as a row that met a bad value is computed again without rounding P.
    ro, rl, to, tl = R.attn_tree(q, kp, vp, table, c, parents, 64 ** -0.5)
    for got, want, tol in ((o, ro, to), (o2, ro, to), (lse, rl, tl), (lse2, rl, tl)):
        R.close(got[:, keep], want[:, keep], tol[:, keep])
    assert not torch.isfinite(o2[:, [1, 4]]).any()


def test_pages_that_are_none():
    """Page numbers outside the pool read as no page, and lengths are kept inside the table."""
    x = list(cache(8, [40, 40, 100, 16], 4, 16, 4, 2, 128, torch.bfloat16))
    x[3][0, 1] = -1
    x[3][1, 0] = x[1].shape[0]
    x[3][2, :] = 2 ** 31 - 1
    check(x, random_parents(9, 4, 4))
    x[4][0], x[4][1], x[4][3] = -7, 10 ** 9, x[3].shape[1] * 16 - 2
    o, lse = check(x, None)
    assert (o[2] == 0).all() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n_draft", [1, 13])
def test_long_context(n_draft, dtype):
    """Few sequences and long contexts: the keys of one row are shared out."""
    x = cache(10, [9000, 1, 4097], n_draft, 64, 8, 2, 128, DT[dtype])
    check(x, random_parents(11, 3, n_draft))
    check(x, None, scale=0.9)


@pytest.mark.parametrize("page", [1, 4, 8, 64, 256])
@pytest.mark.parametrize("Hq,Hkv,n_draft,d", [(8, 2, 24, 128), (8, 2, 40, 128), (6, 2, 43, 64), (3, 1, 64, 128),
                                              (12, 1, 11, 32), (130, 1, 2, 32), (64, 1, 64, 64)])
def test_many_rows(Hq, Hkv, n_draft, d, page):
    """More rows than 64 per key/value head: one query tile, two, and more; short and long."""
    ctx = [0, 3, 127, 128, 700, 4999]
    x = cache(20, ctx, n_draft, page, Hq, Hkv, d, torch.bfloat16)
    check(x, random_parents(21, len(ctx), n_draft, lost=0.1))
    x[3][4, 300 // page] = -1  # a page is missing
    x[3][5, :2 + 2000 // page] = 10 ** 6
    check(x, None)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("n_draft", [20, 40])
def test_many_rows_masked(n_draft, bad):
    """As above with bad values off the path, behind the drafts and in a long chunked row."""
    ctx, page = [5, 250, 4000], 64
    q, kp, vp, table, c = cache(22, ctx, n_draft, page, 8, 2, 128, torch.bfloat16)
    parents = random_parents(23, 3, n_draft)
    parents[:, 1:] = torch.where(parents[:, 1:] == 1, 0, parents[:, 1:])  # nobody descends from draft 1
    used = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
    for n, x in enumerate(ctx):
        for t in range(x + n_draft):
            used[table[n, t // page].long(), t % page] = t != x + 1
    kp, vp = (torch.where(used[:, None, :, None], x, bad) for x in (kp, vp))
    o, lse = api().kda_attn_tree(q, kp, vp, table, c, parents=parents)
    ro, rl, to, tl = R.attn_tree(q, kp, vp, table, c, parents, 128 ** -0.5)
    assert torch.isfinite(ro[:, 2:]).all() and not torch.isfinite(ro[:, 1]).any()
    R.close(o, ro, to)
    R.close(lse, rl, tl)


def test_late_maximum():
    q, kp, vp, table, ctx = cache(12, [3000], 2, 16, 2, 1, 64, torch.bfloat16)
    q[..., 0] = 6.0
    for t in range(3000):
        kp[table[0, t // 16].long(), 0, t % 16, 0] = (t - 1500) / 40
    check((q, kp, vp, table, ctx), None)


def test_runs_are_bit_equal_and_independent_of_the_batch():
    """The same sequence gives the same bits alone, and next to others."""
    x = cache(13, [700, 33, 5000], 9, 32, 8, 2, 128, torch.bfloat16)
    parents = random_parents(14, 3, 9)
    one = api().kda_attn_tree(*x, parents=parents)
    for _ in range(3):
        two = api().kda_attn_tree(*x, parents=parents)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


@pytest.mark.parametrize("n_draft", [1, 9, 24, 50])
def test_calls_one_after_another_agree(n_draft):
    """Many calls without a pause in between, on two sets of inputs in turn."""
    sets = [cache(s, [9000, 130, 4000], n_draft, 64, 8, 2, 128, torch.bfloat16) for s in (25, 26)]
    want = [check(x, None) for x in sets]
    for _ in range(30):
        got = [api().kda_attn_tree(*sets[i % 2]) for i in range(10)]
        for i, (o, lse) in enumerate(got):
            assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_stream_and_graphs():
    attn = api()
    sets = [cache(s, [500, 40], 3, 16, 4, 2, 64, torch.bfloat16) for s in (15, 16)]
    want = [attn.kda_attn_tree(*x) for x in sets]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = attn.kda_attn_tree(*sets[0], stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0][0])
    graphs = []
    for x in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = attn.kda_attn_tree(*x)
        graphs.append((g, r))
    for g, _ in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for (_, r), w in zip(graphs, want):
        assert torch.equal(r[0], w[0]) and torch.equal(r[1], w[1])


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: pages at its end are read where they are."""
    P, Hkv, page, d = 36000, 8, 64, 128  # 2.36e9 elements, 4.7 GB a pool
    kp = torch.zeros(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    g = torch.Generator(device="cuda").manual_seed(17)
    ids = torch.tensor([[P - 1, 3, P - 2]], dtype=torch.int32, device="cuda")
    for i in ids[0].tolist():
        kp[i] = torch.randn(Hkv, page, d, generator=g, device="cuda").to(kp.dtype)
        vp[i] = torch.randn(Hkv, page, d, generator=g, device="cuda").to(kp.dtype)
    q = torch.randn(1, 2, 16, d, generator=g, device="cuda").to(kp.dtype)
    check((q, kp, vp, ids, torch.tensor([170], dtype=torch.int32, device="cuda")), None)


@pytest.mark.parametrize("n_draft", [1, 20, 40])
def test_starved_kernels_report_their_wait(n_draft):
    from gated_delta_rule_132_b200 import kda
    attn = api()
    x = cache(24, [300, 5], n_draft, 16, 8, 2, 128, torch.bfloat16)
    want = attn.kda_attn_tree(*x)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    try:
        kda.kda_debug_set_wait_limit(20000, starve_carry=True)
        attn.kda_attn_tree(*x, workspace=ws)
        status, code = attn.kda_attn_status(ws)
    finally:
        kda.kda_debug_set_wait_limit(0, starve_carry=False)
    assert status == 6 and code != 0
    again = attn.kda_attn_tree(*x, workspace=ws)
    assert attn.kda_attn_status(ws) == (0, 0)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_refusals():
    attn = api()
    from gated_delta_rule_132_b200.kda import KdaError
    q, kp, vp, table, ctx = cache(18, [20, 30], 2, 16, 4, 2, 64, torch.bfloat16)
    with pytest.raises(TypeError):
        attn.kda_attn_tree(q.float(), kp, vp, table, ctx)
    with pytest.raises(ValueError):
        attn.kda_attn_tree(q, kp, vp[:-1], table, ctx)
    with pytest.raises(TypeError):
        attn.kda_attn_tree(q, kp, vp, table.long(), ctx)
    with pytest.raises(ValueError):
        attn.kda_attn_tree(q, kp, vp, table, ctx[:1])
    with pytest.raises(ValueError):
        attn.kda_attn_tree(q, kp, vp, table, ctx, parents=torch.zeros(2, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(KdaError):
        attn.kda_attn_tree(q[:, :, :3].contiguous(), kp, vp, table, ctx)
    with pytest.raises(KdaError):
        attn.kda_attn_tree(q.repeat(1, 40, 1, 1), kp, vp, table, ctx)
    with pytest.raises(ValueError):
        attn.kda_attn_tree(q, kp, vp, table.cpu(), ctx)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n_draft", [1, 9, 20])
def test_batches_of_unequal_lengths(n_draft, dtype):
    """One long sequence among short ones, and more sequences than lengths are added up for."""
    x = cache(31, [20000] + [40 * n for n in range(40)], n_draft, 64, 4, 2, 64, DT[dtype])
    check(x, random_parents(32, 41, n_draft))
    x = cache(33, [(37 * n) % 90 for n in range(1300)], n_draft, 16, 2, 1, 32, DT[dtype], M=300)
    check(x, None)
