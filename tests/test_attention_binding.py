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


def test_workspace_that_is_not_dense():
    """A view with strides covers less memory, or other memory, than its count of elements says."""
    from uncertainty_aware_delta_gb300 import attention

    cpu, made = torch.device("cpu"), []
    buffer = torch.zeros(4096, dtype=torch.uint8)
    assert attention._workspace(buffer, 4096, cpu, made) == (buffer.data_ptr(), 4096)
    assert attention._workspace(buffer.view(torch.int32)[16:], 4000, cpu, made) == (buffer.data_ptr() + 64, 4032)
    for bad in (buffer[:1].expand(4096), buffer[::2], buffer.view(64, 64)[:, :32], buffer.view(64, 64).t()[:32]):
        with pytest.raises(ValueError, match="contiguous"):
            attention._workspace(bad, 512, cpu, made)
    assert not made
