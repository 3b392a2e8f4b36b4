"""Refusals of the full-attention calls at their limits, without a GPU."""
import types

import pytest
import torch

from test_attn_abi import APPEND, COMPACT, FORK, RELEASE, RESERVE, L, at, bwd, call, fwd  # noqa: F401

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("name,defaults", [("kda_cache_fork", FORK), ("kda_cache_reserve", RESERVE),
                                           ("kda_cache_release", RELEASE)])
@pytest.mark.parametrize("P", [MOST, MOST - 8191, MOST - 16383])
def test_pools_whose_page_numbers_end_at_31_bits(L, name, defaults, P):  # noqa: F811
    """A walk over the pages steps beyond the last one, which has to have a number."""
    assert call(L, name, defaults, P=P) == 2


@pytest.mark.parametrize("n", [MOST, MOST - 1023, MOST - 16383])
def test_rows_and_sequences_that_end_at_31_bits(L, n):  # noqa: F811
    for name, defaults in (("kda_cache_reserve", RESERVE), ("kda_cache_release", RELEASE)):
        assert call(L, name, defaults, N=n, M=1) == 2
    assert call(L, "kda_cache_append", APPEND, cu=at(), n=n, B=1, M=1) == 2
    for prompt in (fwd, bwd):
        assert prompt(L, cu=at(), n=n, T=64, Hq=1, Hkv=1) == 2
        assert prompt(L, cu=at(), n=n - 1024, T=1 << 20, Hq=1, Hkv=1) == 2  # its tiles do
    assert L.kda_cache_reserve_workspace_size(n, 1, 4) == 0


@pytest.mark.parametrize("where", [0x10000, 0x20000, 0x20000 + 4 * 3, 0x20000 - 4 * 3, 0x30000 + 4 * 19,
                                   0x10000 + 4 * 31])
def test_compact_does_not_write_lengths_that_it_reads(L, where):  # noqa: F811
    """Rows have several blocks, which all read the old lengths, the path and the table."""
    kw = dict(table=at(0x10000), ctx=at(0x20000), path=at(0x30000))
    assert call(L, "kda_cache_compact", COMPACT, new=at(where), **kw) == 1


def test_streams_of_another_device_are_refused():
    """The work would run on the stream's device with pointers into the inputs'."""
    from gated_delta_rule_132_b200 import attn
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is on cuda:1, expected cuda:0"):
        attn._on(torch.device("cuda", 0), other, lambda: pytest.fail("launched"))


@pytest.mark.parametrize("shape", [(0,), (1,), (3, 0), (2, 3), ()])
def test_offsets_of_another_shape_are_refused(shape):
    """An empty tensor has no address: the call would have taken the tokens as one sequence."""
    from gated_delta_rule_132_b200 import attn
    with pytest.raises(ValueError, match="cu_seqlens must be"):
        attn._sequences(torch.zeros(shape, dtype=torch.int32), torch.device("cuda", 0))


@pytest.mark.parametrize("dtype,chunks", [(0, 32), (1, 16)])
def test_tree_calls_are_planned_for_their_kernel(L, dtype, chunks):  # noqa: F811
    """64 rows per key/value head over 2048 keys: in fp32 chunks of 64 keys at least (two CTAs
    to an SM), in bf16 of 128."""
    R, Hq, Hkv, d = 16, 32, 8, 128
    size = L.kda_attn_tree_workspace_size(1, R, Hq, Hkv, d, 128, 16, dtype)
    assert size == 256 + R * Hq * chunks * (8 + 4 * d)
