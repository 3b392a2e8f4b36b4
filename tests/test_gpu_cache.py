"""The cache's pages against lists, and a whole serving run of the full-attention layer."""
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def api():
    from gated_delta_rule_132_b200 import attn
    return attn


def ints(x):
    return torch.tensor(x, **I32)


def state(seed, N, M, P, page, longest):
    """Rows of random lengths on random pages, as lists and on the device."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, longest + 1, (N,), generator=g).tolist()
    perm = torch.randperm(P, generator=g).tolist()
    refs, table, a = [0] * P, [], 0
    for n in lens:
        c = -(-n // page)
        row = perm[a:a + c]
        a += c
        for p in row:
            refs[p] = 1
        table.append(row + [-1] * (M - c))
    return R.Pages(refs, table, lens, page), ints(refs), ints(table), ints(lens)


def same(model, refs, table, lens):
    assert refs.tolist() == model.refs
    assert table.tolist() == model.table
    assert lens.tolist() == model.lens


@pytest.mark.parametrize("N,M,P,page,longest", [(1, 1, 1, 1, 1), (7, 9, 80, 4, 30), (70, 12, 900, 16, 150),
                                                (1500, 5, 9000, 8, 30), (40, 40, 20001, 64, 2000)])
def test_tables(N, M, P, page, longest):
    """Forks, growth with copies on write, and cuts in a random order."""
    attn = api()
    model, refs, table, lens = state(N, N, M, P, page, longest)
    g = torch.Generator().manual_seed(N + 1)
    for step in range(6):
        parents = torch.randint(-1, N, (N,), generator=g)
        if step % 2:
            parents = torch.arange(N)
            parents[::3] = 0
        table, lens = attn.kda_cache_fork(refs, table, lens, parents.int().cuda())
        model.fork(parents.tolist())
        same(model, refs, table, lens)
        add = torch.randint(0, max(2, page), (N,), generator=g)
        copies, status = attn.kda_cache_reserve(refs, table, lens, add.int().cuda(), page)
        want, code = model.reserve(add.tolist())
        assert status.item() == code and copies.tolist() == want
        same(model, refs, table, lens)
        cut = (lens.cpu() - torch.randint(0, 2 * page, (N,), generator=g)).int()
        attn.kda_cache_release(refs, table, lens, cut.cuda(), page)
        model.release(cut.tolist())
        same(model, refs, table, lens)
    attn.kda_cache_release(refs, table, lens, torch.zeros(N, **I32), page)
    assert not refs.any() and not lens.any() and (table == -1).all()


def test_tables_of_many_rows():
    """More rows than one block's threads, and than it keeps the places of on the chip."""
    test_tables(1500, 5, 9000, 8, 25)
    test_tables(5000, 4, 17000, 16, 40)


def test_reserve_all_or_nothing():
    attn = api()
    refs, table, lens = ints([1, 1, 0, 1]), ints([[0, 3], [1, -1]]), ints([7, 4])
    before = [x.clone() for x in (refs, table, lens)]
    for add, want in (([1, 5], -2), ([0, 4], 0), ([2, 1], -1), ([0, 3], 1)):
        copies, status = attn.kda_cache_reserve(refs, table, lens, ints(add), 4)
        assert status.item() == want
        if want:
            assert all(torch.equal(a, b) for a, b in zip((refs, table, lens), before)) and (copies == -1).all()
        else:
            assert table[1].tolist() == [1, 2] and lens.tolist() == [7, 8] and refs.tolist() == [1, 1, 1, 1]
            lens[1], table[1, 1] = 4, -1  # as before, but for the page that is held
            before = [x.clone() for x in (refs, table, lens)]
    # huge and negative growth
    assert attn.kda_cache_reserve(refs, table, lens, ints([0, 2 ** 31 - 1]), 4)[1].item() == -2
    assert attn.kda_cache_reserve(refs, table, lens, ints([-5, -2 ** 31]), 4)[1].item() == 0
    assert all(torch.equal(a, b) for a, b in zip((refs, table, lens), before))


def test_fork_grows_and_shrinks_the_batch():
    attn = api()
    model, refs, table, lens = state(3, 5, 6, 40, 8, 40)
    for parents in ([0, 0, 0, 4, 2, 2, 9, -1, -7], [8, 3], [0, 1, 1]):
        table, lens = attn.kda_cache_fork(refs, table, lens, ints(parents))
        model.fork(parents)
        same(model, refs, table, lens)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hkv,page,d", [(1, 1, 32), (3, 16, 64), (8, 64, 128), (2, 1024, 32)])
def test_copy_pages(Hkv, page, d, dtype):
    attn, P = api(), 12
    kp, vp = (torch.randn(P, Hkv, page, d, device="cuda").to(dtype) for _ in range(2))
    # dropped: bad numbers, a second destination 5, a destination that is a source, itself
    pairs = [(0, 5), (-1, -1), (1, 5), (2, 6), (2, 7), (9, 0), (3, 12), (-4, 3), (4, 4), (11, 10)]
    want = [x.clone() for x in (kp, vp)]
    for w in want:
        for a, b in ((0, 5), (2, 6), (2, 7), (11, 10)):
            w[b] = w[a]
    attn.kda_cache_copy_pages(kp, vp, ints(pairs))
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hkv,page,d", [(1, 1, 32), (3, 16, 64), (8, 32, 128)])
def test_append_and_compact(Hkv, page, d, dtype):
    attn, n_draft = api(), 9
    start = [0, 3, page, 2 * page - 1, 30, 31]
    N, M = len(start), -(-(max(start) + n_draft) // page) + 1
    P = N * M + 1
    kp, vp = (torch.randn(P, Hkv, page, d, device="cuda").to(dtype) for _ in range(2))
    table = torch.randperm(P - 1, device="cuda")[:N * M].view(N, M).int().contiguous()
    table[4, (start[4] + 2) // page] = -1  # one page is missing
    new = [torch.randn(N, n_draft, Hkv, d, device="cuda").to(dtype) for _ in range(2)]
    want = [x.clone() for x in (kp, vp)]
    put = lambda w, n, pos: (w, table[n, pos // page].item(), pos % page)  # noqa: E731
    for w, x in zip(want, new):
        for n in range(N):
            for i in range(n_draft):
                _, p, slot = put(w, n, start[n] + i)
                if p >= 0:
                    w[p, :, slot] = x[n, i]
    attn.kda_cache_append(kp, vp, table, ints(start), *new)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    paths = [list(range(n_draft)), [-1] * n_draft, [8] + [-1] * 8, [0, 2, 3, 7, 8, -1, 9, 1, 1],
             [1, 3, 4, 6, 7, 8, -1, -1, -1], [2, 5, 5, 6, 7, 8, 8, 8, 8]]
    kept = [9, 0, 1, 5, 6, 2]
    for w in want:
        for n in range(N):
            for j, i in enumerate(paths[n][:kept[n]]):
                _, a, sa = put(w, n, start[n] + i)
                _, b, sb = put(w, n, start[n] + j)
                if a >= 0 and b >= 0:
                    w[b, :, sb] = w[a, :, sa].clone()
    lens = attn.kda_cache_compact(kp, vp, table, ints(start), ints(paths))
    assert lens.tolist() == [s + k for s, k in zip(start, kept)]
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_append_packed_and_outside():
    """Packed prompts of odd lengths; positions before the row or behind its table are left out."""
    attn, page, Hkv, d = api(), 8, 2, 64
    lens, start = [5, 0, 17, 1], [0, 4, -3, 30]
    cu = ints([0, 5, 5, 22, 23])
    T = 26  # three tokens belong to nobody
    table = torch.randperm(16, device="cuda").view(4, 4).int().contiguous()
    kp, vp = (torch.zeros(16, Hkv, page, d, device="cuda") for _ in range(2))
    kn, vn = (torch.randn(1, T, Hkv, d, device="cuda") for _ in range(2))
    want = torch.zeros_like(kp)
    for n, (c, s) in enumerate(zip(lens, start)):
        for i in range(c):
            if s >= 0 and s + i < 32:
                want[table[n, (s + i) // page].long(), :, (s + i) % page] = kn[0, cu[n] + i]
    attn.kda_cache_append(kp, vp, table, ints(start), kn, vn, cu_seqlens=cu)
    assert torch.equal(kp, want)
    attn.kda_cache_append(kp, vp, table, ints([2 ** 31 - 1] * 4), kn, vn, cu_seqlens=cu)
    assert torch.equal(kp, want)


def test_refusals():
    attn = api()
    from gated_delta_rule_132_b200.kda import KdaError
    refs, table, lens = ints([1, 0]), ints([[0, -1]]), ints([3])
    with pytest.raises(TypeError):
        attn.kda_cache_fork(refs, table, lens, torch.zeros(1, device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError):
        attn.kda_cache_reserve(refs, table, ints([3, 4]), ints([1]), 4)
    with pytest.raises(KdaError):
        attn.kda_cache_reserve(refs, table, lens, ints([1]), 5)
    with pytest.raises(ValueError):
        attn.kda_cache_release(refs, table.t(), lens, ints([1]), 4)
    kp = torch.zeros(2, 1, 4, 32, device="cuda")
    with pytest.raises(ValueError):
        attn.kda_cache_append(kp, kp, table, ints([0]), torch.zeros(2, 1, 1, 32, device="cuda"), kp[:, :, :1])
    with pytest.raises(ValueError):
        attn.kda_cache_compact(kp, kp, table, ints([0]), ints([1]))
    with pytest.raises(ValueError):
        attn.kda_cache_copy_pages(kp, kp, ints([[0, 1, 2]]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_serving_run(dtype):
    """Prompts, a fork, three rounds of drafted trees with some accepted, and a release: every
    token's output is that of attention over the tokens its sequence has kept."""
    attn, Hq, Hkv, d, page, n_draft = api(), 4, 2, 64, 16, 5
    g = torch.Generator(device="cuda").manual_seed(31)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    lens0 = [37, 16, 3]
    cu = ints([0, 37, 53, 56])
    q, k, v = mk(1, 56, Hq, d), mk(1, 56, Hkv, d), mk(1, 56, Hkv, d)
    o, lse = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu)
    ro, rl, to, tl = R.attn_fwd(q[0], k[0], v[0], [(0, 37), (37, 16), (53, 3)], d ** -0.5)
    R.close(o[0], ro, to)
    P, M = 60, 8
    kp, vp = (torch.full((P, Hkv, page, d), float("nan"), device="cuda").to(dtype) for _ in range(2))
    refs, table, lens = torch.zeros(P, **I32), torch.full((3, M), -1, **I32), torch.zeros(3, **I32)
    _, status = attn.kda_cache_reserve(refs, table, lens, ints(lens0), page)
    assert status.item() == 0
    attn.kda_cache_append(kp, vp, table, torch.zeros(3, **I32), k, v, cu_seqlens=cu)
    table, lens = attn.kda_cache_fork(refs, table, lens, ints([0, 0, 1, 2, 0]))
    rows = [0, 0, 1, 2, 0]
    kept = [[(k[0, cu[r]:cu[r + 1]]), (v[0, cu[r]:cu[r + 1]])] for r in rows]
    N = 5
    parents = ints([[-1, 0, 0, 1, 2]] * N)
    for step in range(3):
        qn, kn, vn = mk(N, n_draft, Hq, d), mk(N, n_draft, Hkv, d), mk(N, n_draft, Hkv, d)
        ctx = lens.clone()
        copies, status = attn.kda_cache_reserve(refs, table, lens, torch.full((N,), n_draft, **I32), page)
        assert status.item() == 0
        attn.kda_cache_copy_pages(kp, vp, copies)
        attn.kda_cache_append(kp, vp, table, ctx, kn, vn)
        o, lse = attn.kda_attn_tree(qn, kp, vp, table, ctx, parents=parents)
        for n in range(N):
            for i, path in enumerate([[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4]]):
                kk, vv = (torch.cat([a, b[n, path]]) for a, b in zip(kept[n], (kn, vn)))
                see = torch.ones(1, kk.shape[0], dtype=torch.bool, device="cuda")
                for h in range(Hq):
                    ro, rl, to, tl = R.attend(qn[n, i, h][None].double(), kk[:, h // 2].double(),
                                              vv[:, h // 2].double(), see, d ** -0.5, dtype)
                    R.close(o[n, i, h][None], ro, to)
                    R.close(lse[n, i, h][None], rl, tl)
        paths = [[0, 2, 4], [0, 1], [], [0], [0, 1, 3]]
        path = ints([p + [-1] * (n_draft - len(p)) for p in paths])
        new_lens = attn.kda_cache_compact(kp, vp, table, ctx, path)
        attn.kda_cache_release(refs, table, lens, new_lens, page)
        for n, p in enumerate(paths):
            kept[n] = [torch.cat([a, b[n, p]]) for a, b in zip(kept[n], (kn, vn))]
        assert lens.tolist() == [x[0].shape[0] for x in kept]
    attn.kda_cache_release(refs, table, lens, torch.zeros(N, **I32), page)
    assert not refs.any()
