"""The prompt forward's kernel source on the host (tests/cuda_host/tc_emu): its warps go on in
orders drawn from seeds, each as late as it can be after any arrival, copies land in any order
and products when the scheduler takes them. Results against the fp64 form, and no wait may run
out in any order."""
import ctypes

import pytest
import torch

import attn_ref as R
import host_kernels


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return host_kernels.build(tmp_path_factory.mktemp("attn_fwd"), ("kda_attn_fwd.cu",), "attn_fwd_host.cpp")


def inputs(seed, T, Hq, Hkv, d):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, h, d, generator=g).bfloat16() for h in (Hq, Hkv, Hkv)]


def spans_of(lens):
    ends = torch.tensor(lens).cumsum(0).tolist()
    return [(e - n, n) for e, n in zip(ends, lens)]


def run(host, x, lens, packed, ctas, seed, spare=0):
    """One call on `ctas` CTAs: o and lse; `spare` tokens lie behind the last sequence."""
    q, k, v = x
    T, Hq, d = q.shape
    o, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0)
    cu = torch.tensor([0] + [a + n for a, n in spans_of(lens)], dtype=torch.int32)
    ws = torch.zeros(1 << 18, dtype=torch.uint8)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    status = host.attn_fwd_host_run(p(q), p(k), p(v), p(cu) if packed else None, len(lens),
                                    1 if packed else len(lens), T if packed else lens[0], Hq, k.shape[1], d,
                                    ctypes.c_float(d ** -0.5), p(o), p(lse), p(ws), ctas, ctypes.c_uint(seed))
    assert status == 0, f"a wait ran out: {status}"
    if spare:
        assert (o[-spare:] == 7.0).all() and (lse[-spare:] == 7.0).all()
    return o, lse


def check(got, x, lens):
    ro, rl, to, tl = R.attn_fwd(*x, spans_of(lens), x[0].shape[2] ** -0.5)
    R.close(got[0], ro, to)
    R.close(got[1], rl, tl)


@pytest.mark.parametrize("lens,packed,Hq,Hkv,d,ctas", [
    ([100, 130, 20], True, 2, 1, 32, 1),     # items of two heads, one after another on a CTA
    ([300, 130, 5, 0, 64], True, 1, 1, 64, 1),  # of two tiles of a head, and of one
    ([1] * 9, True, 4, 2, 64, 1),            # as short as can be
    ([260, 260], False, 1, 1, 128, 1),
    ([140] * 3, False, 2, 1, 128, 2),
])
def test_any_order(host, lens, packed, Hq, Hkv, d, ctas):
    x = inputs(1, sum(lens), Hq, Hkv, d)
    first = None
    for seed in range(12):
        got = run(host, x, lens, packed, ctas, 100 * seed)
        if first is None:
            check(got, x, lens)
            first = got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("heads", [1, 2])
def test_moving_reference(host, heads):
    """Scores that rise towards a sequence's first key, so that the last step rescales too."""
    lens = [256, 200]
    q, k, v = inputs(2, sum(lens), heads, 1, 32)
    q[..., 0] = 6.0
    for a, n in spans_of(lens):
        k[a:a + n, 0, 0] = torch.linspace(40, -40, n).bfloat16()
    for seed in range(8):
        check(run(host, (q, k, v), lens, True, 1, 50 * seed), (q, k, v), lens)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq,Hkv,d,lens", [(2, 1, 32, [30, 150]), (1, 1, 128, [300]), (1, 1, 64, [70]),
                                           (16, 1, 32, [140]), (6, 3, 128, [140])])  # one such item after another
def test_padding_takes_no_other_way(host, Hq, Hkv, d, lens, bad):
    """What lies behind the last sequence changes no bit: no row is computed again because of it."""
    spare = 60
    q, k, v = inputs(3, sum(lens) + spare, Hq, Hkv, d)
    for seed in range(8):
        want = run(host, (q, k, v), lens, True, 1, 10 * seed, spare)
        x = [t.clone() for t in (q, k, v)]
        for t in x:
            t[-spare:] = bad
        got = run(host, x, lens, True, 1, 10 * seed, spare)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
