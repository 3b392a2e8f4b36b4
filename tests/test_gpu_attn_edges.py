"""Full attention and its cache where calls meet, end or are padded: bounds from attn_ref."""
import pytest
import torch

import attn_ref as R
from test_gpu_attn import api, cu_of, inputs, spans_of
from test_gpu_attn_tree import cache, random_parents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv", [(16, 8), (16, 16)])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_many_short_items_follow_one_another(d, Hq, Hkv):
    """Items of one or two steps, ten to a CTA, whose products follow one another closely: no
    wait runs out in any of the calls, and all give the same bits."""
    attn = api()
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(1, 200, (200,), generator=g).tolist()
    q, k, v, _ = inputs(40, sum(lens), Hq, Hkv, d, torch.bfloat16)
    cu, ws = cu_of(lens), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    o, lse = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu, workspace=ws)
    assert attn.kda_attn_status(ws) == (0, 0)
    ro, rl, to, tl = R.attn_fwd(q[0], k[0], v[0], spans_of(lens), d ** -0.5)
    R.close(o[0], ro, to)
    R.close(lse[0], rl, tl)
    for _ in range(50):
        again = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu, workspace=ws)
        assert attn.kda_attn_status(ws) == (0, 0)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64), (2, 2, 32)])
def test_padding_takes_no_other_way(Hq, Hkv, d, bad, dtype):
    """Tokens behind the last sequence, and what nobody wrote into their o and lse, change no bit
    of the others' results: no row is computed again because of them. (A row that is computed
    again rounds no probability to 16 bits, so its bits differ.)"""
    attn, lens, spare = api(), [257, 1000], 70
    T = sum(lens) + spare
    x = inputs(41, T, Hq, Hkv, d, dtype)
    cu = cu_of(lens)

    def run(q, k, v, dO, fill):
        o, lse = torch.full_like(q, fill), torch.full((1, T, Hq), fill, device="cuda")
        attn.kda_attn_fwd(q, k, v, cu_seqlens=cu, o=o, lse=lse)
        g = attn.kda_attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu)
        return [t[:, :-spare] for t in (o, lse, *g.values())]

    want = run(*x, 0.0)
    for which in ([0, 1, 2, 3], [3], []):
        y = [t.clone() for t in x]
        for i in which:
            y[i][:, -spare:] = bad
        assert all(torch.equal(a, b) for a, b in zip(run(*y, bad), want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sequences_that_are_all_empty(dtype):
    """Nothing is written, and calls with tokens on the same workspace are as they would be alone."""
    attn, T = api(), 150
    q, k, v, dO = inputs(42, T, 4, 2, 64, dtype)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    none, cu = torch.zeros(3, dtype=torch.int32, device="cuda"), cu_of([100, 50])
    want = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu)
    grads = attn.kda_attn_bwd(q, k, v, *want, dO, cu_seqlens=cu)
    o, lse = torch.full_like(q, 7.0), torch.full((1, T, 4), 7.0, device="cuda")
    for _ in range(20):
        attn.kda_attn_fwd(q, k, v, cu_seqlens=none, workspace=ws, o=o, lse=lse)
        attn.kda_attn_bwd(q, k, v, o, lse, dO, cu_seqlens=none, workspace=ws)
        got = attn.kda_attn_bwd(q, k, v, *want, dO, cu_seqlens=cu, workspace=ws)
        assert all(torch.equal(got[n], grads[n]) for n in grads)
    assert attn.kda_attn_status(ws) == (0, 0)
    assert (o == 7.0).all() and (lse == 7.0).all()


def test_offsets_of_another_shape_are_refused():
    attn = api()
    q, k, v, dO = inputs(43, 8, 2, 1, 64, torch.bfloat16)
    o, lse = attn.kda_attn_fwd(q, k, v)
    kp = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    for shape in ((0,), (1,), (3, 0), (2, 3), ()):
        cu = torch.zeros(shape, dtype=torch.int32, device="cuda")
        for call in (lambda: attn.kda_attn_fwd(q, k, v, cu_seqlens=cu),
                     lambda: attn.kda_attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu),
                     lambda: attn.kda_cache_append(kp, kp, one[None], one, k, v, cu_seqlens=cu)):
            with pytest.raises(ValueError, match="cu_seqlens must be"):
                call()


def sanitised(offsets, T):
    """(start, length) of every sequence as the prompt calls take malformed offsets."""
    starts, most = [], 0
    for x in offsets:
        most = max(most, min(max(x, 0), T))
        starts.append(most)
    return [(a, b - a) for a, b in zip(starts, starts[1:])]


@pytest.mark.parametrize("dtype,Hkv,d", [(torch.bfloat16, 2, 128), (torch.float32, 1, 32), (torch.bfloat16, 1, 32)])
@pytest.mark.parametrize("offsets,T", [
    ([0, 90, 40, 400], 200), ([-5, 20, 200], 200), ([7, 7, 3, 150, 150], 160), ([300, 400], 200), ([-9, -2], 50),
    (list(range(0, 3000, 5)) + [10, -1, 2996], 3000),   # more offsets than a block's threads
    (list(range(2, 1026)), 1100), (list(range(2, 1027)), 1100),  # at the border of many sequences
    ([0] * 1600 + [64, 0, 1000, 5, 900, 2000], 1500),
    ([0, 900, 100] * 6000 + [2000, 1900, 2100], 2500),  # several looks
    ([0, 12345, 12346, 40000], 40000),
])
def test_append_takes_offsets_as_the_prompt_does(offsets, T, dtype, Hkv, d):
    """Falling, negative and too large offsets: each token at the position that the attention of
    the same prompt gives it."""
    attn, page, spans = api(), 16, sanitised(offsets, T)
    N, longest = len(spans), max(n for _, n in spans)
    start = torch.arange(N, device="cuda", dtype=torch.int32) % 5
    M = -(-(longest + 5) // page)
    owners = [n for n, (_, count) in enumerate(spans) if count]
    table = torch.full((N, M), -1, dtype=torch.int32, device="cuda")
    for i, n in enumerate(owners):
        table[n] = torch.arange(i * M, (i + 1) * M, device="cuda")
    pools = [torch.zeros(max(len(owners), 1) * M, Hkv, page, d, dtype=dtype, device="cuda") for _ in range(2)]
    new = [torch.randn(1, T, Hkv, d, device="cuda").to(dtype) for _ in range(2)]
    want = [x.clone() for x in pools]
    for n in owners:
        a, count = spans[n]
        pos = torch.arange(count, device="cuda") + start[n]
        for w, x in zip(want, new):
            w[table[n][pos // page].long(), :, pos % page] = x[0, a:a + count]
    attn.kda_cache_append(*pools, table, start, *new,
                          cu_seqlens=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1])


def test_copies_of_more_rows_than_one_call_takes():
    """20000 rows that share their last pages in twos: each pair's second holder gets the page, the
    first a copy, with the pairs handed over in parts."""
    attn, N, page = api(), 20000, 4
    i32 = dict(dtype=torch.int32, device="cuda")
    P = N // 2 * 3
    refs, lens = torch.zeros(P, **i32), torch.full((N,), 3, **i32)
    refs[:N // 2] = 2
    table = torch.full((N, 2), -1, **i32)
    table[:, 0] = torch.arange(N, device="cuda") // 2
    kp, vp = (torch.randn(P, 1, page, 32, device="cuda") for _ in range(2))
    want = [x.clone() for x in (kp, vp)]
    copies, status = attn.kda_cache_reserve(refs, table, lens, torch.ones(N, **i32), page)
    assert status.item() == 0 and (lens == 4).all()
    for part in copies.split(16384):
        attn.kda_cache_copy_pages(kp, vp, part)
    made = copies[::2]
    assert (copies[1::2] == -1).all()
    assert torch.equal(made[:, 0], torch.arange(N // 2, **i32))
    assert torch.equal(made[:, 1], torch.arange(N // 2, N, **i32))
    for w in want:
        w[N // 2:N] = w[:N // 2]
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


@pytest.mark.parametrize("C", [1, 100, 129, 300, 9000, 16384])
def test_copies_in_lists_of_all_lengths(C):
    """However many slices a page gets: pairs that are left out among pairs that are not."""
    attn, P = api(), 2 * 16384 + 8
    kp, vp = (torch.randn(P, 2, 64, 32, device="cuda").bfloat16() for _ in range(2))
    order = torch.randperm(P, generator=torch.Generator().manual_seed(C))
    src, dst = order[:C], order[C:2 * C].clone()
    if C > 2:
        dst[C - 1] = dst[0]  # an earlier pair's destination
        dst[1] = src[2]      # another pair's source
    real = torch.ones(C, dtype=torch.bool)
    if C > 2:
        real[[1, C - 1]] = False
    want = [x.clone() for x in (kp, vp)]
    for w in want:
        w[dst[real].cuda()] = w[src[real].cuda()]
    attn.kda_cache_copy_pages(kp, vp, torch.stack([src, dst], 1).int().cuda().contiguous())
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


# Relative L2 error of a whole result. In bf16 each term of a sum has one rounded factor and the
# sum is rounded once: relative errors of at most u = 2^-8, evenly spread over +-u of a value in
# [1, 2) at worst, so u / sqrt(3) in the mean square, and independent of one another. Terms whose
# signs are independent keep that share in their sum. Two such roundings: u sqrt(2 / 3) = 0.0032;
# the bound leaves a quarter for chance and fp32. In fp32 a score's bound (2 d e sum |q k| scale,
# some 2e-5 here) leads. A group of 16 keys left out of 1500 would show as 0.1.
L2 = {torch.bfloat16: 0.004, torch.float32: 2e-5}


def l2(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,packed", [([1500], False), ([700, 13, 260, 1100], True)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64), (2, 2, 32)])
def test_whole_results(Hq, Hkv, d, lens, packed, dtype):
    attn, spans = api(), spans_of(lens)
    q, k, v, dO = inputs(44, sum(lens), Hq, Hkv, d, dtype)
    cu = cu_of(lens) if packed else None
    o, lse = attn.kda_attn_fwd(q, k, v, cu_seqlens=cu)
    want = R.attn_fwd(q[0], k[0], v[0], spans, d ** -0.5)
    assert l2(o[0], want[0]) <= L2[dtype]
    g = attn.kda_attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu)
    grads, _ = R.attn_bwd(q[0], k[0], v[0], o[0], lse[0], dO[0], spans, d ** -0.5)
    for name, w in zip(("dq", "dk", "dv"), grads):
        assert l2(g[name][0], w) <= L2[dtype], name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_draft", [1, 4, 8, 24, 50])
def test_whole_tree_results_and_the_batch(n_draft, dtype):
    """A whole call, and each of its sequences alone: the split of the keys goes by the batch, so
    bits may differ, but all are within the bounds."""
    q, kp, vp, table, ctx = cache(45, [3000, 33, 700, 1024], n_draft, 32, 8, 2, 128, dtype)
    parents = random_parents(46, 4, n_draft)
    o, lse = api().kda_attn_tree(q, kp, vp, table, ctx, parents=parents)
    ro, rl, to, tl = R.attn_tree(q, kp, vp, table, ctx, parents, 128 ** -0.5)
    assert l2(o, ro) <= L2[dtype]
    for n in range(4):
        part = slice(n, n + 1)
        alone = api().kda_attn_tree(q[part], kp, vp, table[part], ctx[part], parents=parents[part])
        R.close(alone[0], ro[part], to[part])
        R.close(alone[1], rl[part], tl[part])
        assert l2(alone[0], ro[part]) <= L2[dtype] * 1.5  # of one sequence, whose rows are few
