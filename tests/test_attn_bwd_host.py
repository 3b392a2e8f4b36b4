"""The prompt gradients' kernel source on the host, as test_attn_fwd_host runs the forward's."""
import ctypes

import pytest
import torch

import attn_ref as R
import host_kernels
from test_attn_fwd_host import spans_of


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return host_kernels.build(tmp_path_factory.mktemp("attn_bwd"), ("kda_attn_bwd.cu",), "attn_bwd_host.cpp")


def inputs(seed, lens, Hq, Hkv, d, spare=0):
    """q, k, v, o, lse, dO with `spare` tokens behind the last sequence."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + spare
    q, k, v, dO = (torch.randn(T, h, d, generator=g).bfloat16() for h in (Hq, Hkv, Hkv, Hq))
    o, lse = R.attn_fwd(q, k, v, spans_of(lens), d ** -0.5)[:2]
    return q, k, v, o.bfloat16(), lse.float(), dO


def run(host, x, lens, packed, ctas, seed):
    """One call on `ctas` CTAs: dq, dk, dv."""
    q, k = x[:2]
    T, Hq, d = q.shape
    out = [torch.full_like(t, 7.0) for t in x[:3]]
    cu = torch.tensor([0] + [a + n for a, n in spans_of(lens)], dtype=torch.int32)
    ws = torch.zeros(1 << 18, dtype=torch.uint8)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    status = host.attn_bwd_host_run(*map(p, x), p(cu) if packed else None, len(lens), 1 if packed else len(lens),
                                    T if packed else lens[0], Hq, k.shape[1], d, ctypes.c_float(d ** -0.5),
                                    *map(p, out), p(ws), ctas, ctypes.c_uint(seed))
    assert status == 0, f"a wait ran out: {status}"
    return out


@pytest.mark.parametrize("lens,packed,H,d,ctas", [
    ([100, 130, 20], True, 2, 32, 1),
    ([300, 5, 0, 64], True, 1, 64, 1),
    ([1] * 5, True, 2, 64, 1),
    ([140] * 2, False, 1, 128, 2),
])
def test_any_order(host, lens, packed, H, d, ctas):
    x = inputs(1, lens, H, H, d)
    want, tol = R.attn_bwd(*x, spans_of(lens), d ** -0.5)
    first = None
    for seed in range(6):
        got = run(host, x, lens, packed, ctas, 1000 * seed)
        if first is None:
            first = got
            for g, w, t in zip(got, want, tol):
                R.close(g, w, t)
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d,lens", [(32, [30, 150]), (128, [200]), (64, [70])])
def test_padding_takes_no_other_way(host, d, lens, bad):
    """What lies behind the last sequence changes no bit: no row is computed again because of it."""
    spare = 60
    x = inputs(3, lens, 1, 1, d, spare)
    for seed in range(3):
        want = run(host, x, lens, True, 1, 10 * seed)
        for what in (range(6), [3, 4], [5], [0, 1, 2]):  # all, o and lse that nobody wrote, dO, q k v
            y = [t.clone() for t in x]
            for i in what:
                y[i][-spare:] = bad
            got = run(host, y, lens, True, 1, 10 * seed)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((t[-spare:] == 7.0).all() for t in got)
