"""Tree attention of many rows: its kernel's source on the host, as test_attn_fwd_host runs the
forward's, with the plan, the join and the host side around it."""
import ctypes

import pytest
import torch

import attn_ref as R
import host_kernels


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return host_kernels.build(tmp_path_factory.mktemp("attn_tree"), ("kda_attn_tree.cu", "kda_attn_tree_tc.cu"),
                              "attn_tree_host.cpp", "attn_tree_tc_host.cpp")


def inputs(seed, ctx, n_draft, page, Hq, Hkv, d):
    g = torch.Generator().manual_seed(seed)
    need = [-(-(c + n_draft) // page) for c in ctx]
    P, M = sum(need) + 2, max(need)
    perm = torch.randperm(P, generator=g).int()
    table = torch.full((len(ctx), M), -1, dtype=torch.int32)
    a = 0
    for n, c in enumerate(need):
        table[n, :c] = perm[a:a + c]
        a += c
    mk = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    parents = torch.stack([torch.tensor([-1] + [int(torch.randint(-1, i, (1,), generator=g)) for i in range(1, n_draft)])
                           for _ in ctx]).int()
    return (mk(len(ctx), n_draft, Hq, d), mk(P, Hkv, page, d), mk(P, Hkv, page, d), table,
            torch.tensor(ctx, dtype=torch.int32), parents)


def run(host, x, seed):
    q, kp, vp, table, ctx, parents = x
    N, n_draft, Hq, d = q.shape
    P, Hkv, page, _ = kp.shape
    o, lse = torch.full_like(q, 7.0), torch.full((N, n_draft, Hq), 7.0)
    ws = torch.zeros(1 << 24, dtype=torch.uint8)
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    status = host.attn_tree_host_run(p(q), p(kp), p(vp), p(table), p(ctx), p(parents), N, n_draft, Hq, Hkv, d, P,
                                     table.shape[1], page.bit_length() - 1, ctypes.c_float(d ** -0.5), p(o), p(lse),
                                     p(ws), ctypes.c_ulonglong(ws.numel()), ctypes.c_uint(seed))
    assert status == 0, f"a wait ran out, or the call: {status}"
    return o, lse


@pytest.mark.parametrize("ctx,n_draft,page,Hq,Hkv,d", [
    ([300], 40, 16, 1, 1, 32),          # one query tile, keys in halves; chunks
    ([3, 0], 20, 64, 2, 1, 64),         # a sequence with drafts only
    ([140], 64, 8, 3, 1, 32),           # two query tiles
    ([130], 33, 2, 4, 1, 128),          # two, pages too small for boxes
    ([700], 11, 128, 12, 1, 32),
])
def test_any_order(host, ctx, n_draft, page, Hq, Hkv, d):
    x = inputs(1, ctx, n_draft, page, Hq, Hkv, d)
    want = R.attn_tree(*x, d ** -0.5)
    first = None
    for seed in range(4):
        got = run(host, x, 1000 * seed)
        if first is None:
            R.close(got[0], want[0], want[2])
            R.close(got[1], want[1], want[3])
            first = got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("n_draft", [20, 40])
def test_bad_values_off_the_path(host, n_draft):
    ctx, page = [70, 5], 64
    q, kp, vp, table, c, parents = inputs(2, ctx, n_draft, page, 4, 1, 32)
    parents[:, 1:] = torch.where(parents[:, 1:] == 1, 0, parents[:, 1:])  # nobody descends from draft 1
    used = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    for n, x in enumerate(ctx):
        for t in range(x + n_draft):
            used[table[n, t // page].long(), t % page] = t != x + 1
    kp, vp = (torch.where(used[:, None, :, None], x, float("nan")) for x in (kp, vp))
    x = (q, kp, vp, table, c, parents)
    want = R.attn_tree(*x, 32 ** -0.5)
    for seed in range(2):
        got = run(host, x, seed)
        R.close(got[0], want[0], want[2])
        R.close(got[1], want[1], want[3])
