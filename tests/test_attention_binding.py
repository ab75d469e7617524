"""Checks of the attention binding that need no GPU: arguments are refused before anything is enqueued."""
import pytest
import torch

from test_attention_abi import lib  # noqa: F401

BIG = [2 ** 31, 2 ** 32, 2 ** 32 + 16, -2 ** 31 - 1, 2 ** 40]


def _calls():
    import uncertainty_aware_delta_gb300 as kdn

    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    cache, table = torch.zeros(3, 2, 1, 18 * 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.int32)
    return {
        "window": [lambda n: kdn.kdn_prompt_attention(x, x, x, i, window=n),
                   lambda n: kdn.kdn_cache_attention(x, cache, table, i, window=n),
                   lambda n: kdn.cache_attention_workspace_size(4, 2, 2, 64, 100, n)],
        "max_len": [lambda n: kdn.kdn_cache_attention(x, cache, table, i, max_len=n),
                    lambda n: kdn.cache_attention_workspace_size(4, 2, 2, 64, n)],
        "page": [lambda n: kdn.kdn_cache_plan(i, i, table, i, i[:1], page=n, capacity=8), lambda n: kdn.cache_alloc(3, n, 2, 64, "cpu")],
        "capacity": [lambda n: kdn.kdn_cache_plan(i, i, table, i, i[:1], page=16, capacity=n, out=[i] * 6)],
        "flags": [lambda n: kdn.kdn_prompt_attention(x, x, x, i, flags=n),
                  lambda n: kdn.prompt_attention_workspace_size(4, 4, 2, 2, 64, flags=n)],
        "total_q": [lambda n: kdn.prompt_attention_workspace_size(4, n, 2, 2, 64)],
    }


@pytest.mark.parametrize("name", ["window", "max_len", "page", "capacity", "flags", "total_q"])
def test_numbers_past_32_bits(lib, name):  # noqa: F811
    """ctypes would cut them off to 32 bits: a window of 2^32 to none."""
    for call in _calls()[name]:
        for n in BIG:
            with pytest.raises(ValueError, match=name):
                call(n)
