"""Limits of the attention's calls on the host, beside those of test_attention_abi.py."""
import pytest
import torch

from test_attention_abi import ARG, B16, DEVICE, NO_GPU, SIZE, a, call, made  # noqa: F401 (a, made: fixtures)


@pytest.mark.parametrize("name", ["hc_attend", "hc_attend_shared"])
def test_positions_that_32_bits_cannot_count_are_refused(a, name):
    """Tables of 2^31 positions, for which the last unit's end is no 32-bit number; with its prefix, a sequence counts as
    one."""
    wide = lambda own, pre: {"cache.page_size": 65536, "batch.width": own, "batch.table_row": own, "prefix.width": pre, "prefix.table_row": pre}  # noqa: E731
    both = name == "hc_attend_shared"
    for own, pre in [(32768, 5), (40000, 5)] + ([(5, 32768), (16384, 16384), (32767, 1)] if both else []):
        assert call(a, name, **wide(own, pre)) == SIZE, (own, pre)
    if NO_GPU:
        for own, pre in [(32767, 0), (5, 5)] + ([(16384, 16383), (1, 32766)] if both else []):
            assert call(a, name, **wide(own, pre)) == DEVICE, (own, pre)


@pytest.mark.parametrize("T", [0, 1, 5])
def test_no_heads_are_taken_for_any_number_of_tokens(a, made, T):
    """(The calls then refuse the CPU's tensors, which is their last check.)"""
    cache, batch, _ = made
    none, k = torch.zeros((T, 0, 64), dtype=B16), torch.zeros((T, 2, 64), dtype=B16)
    for run in (lambda: a.rotate_heads(none), lambda: a.rotate_heads(none, out=none.clone()), lambda: a.append_heads(none, k, k, cache, batch),
                lambda: a.append_heads(k[:, 1:1], k, k, cache, batch)):
        with pytest.raises(ValueError, match="GPU"):
            run()
    with pytest.raises(ValueError, match="multiple of the cache's"):
        a.attend(none, cache, batch)


def test_types_that_differ_from_the_caches_are_refused(a, made):
    cache, batch, prefix = made
    q, k, p = torch.zeros((4, 8, 64), dtype=B16), torch.zeros((4, 2, 64), dtype=B16), torch.zeros(4, dtype=torch.int32)
    for run in (lambda: a.append_heads(q.half(), k, k, cache, batch), lambda: a.append_heads(q.float(), k, k, cache, batch),
                lambda: a.append_heads(q, k, k.half(), cache, batch), lambda: a.append_heads(None, k.half(), k.half(), cache, batch),
                lambda: a.append_heads(q, k, k, cache, batch, out=q.half()), lambda: a.append_heads(q, k, k, cache, batch, positions=p.short()),
                lambda: a.attend(q.half(), cache, batch), lambda: a.attend(q, cache, batch, out=q.half()),
                lambda: a.attend_shared(q.half(), cache, batch, prefix), lambda: a.attend_shared(q, cache, batch, prefix, last=p.long())):
        with pytest.raises(TypeError):
            run()
