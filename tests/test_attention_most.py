"""Counts near 2^31 that the kernels' loops and grids cannot step past: refused on the host, so no GPU is needed."""
import pytest

from test_attention_abi import MB, lib, vp  # noqa: F401

MOST = 2 ** 31 - 1 - 2 ** 25


@pytest.mark.parametrize("what", ["n", "nq", "nk"])
def test_prompt_counts(lib, what):  # noqa: F811
    def call(n=2, nq=40, nk=40):
        return lib.kdn_prompt_attention(n, nq, nk, 1, 1, 16, 0, 0.0, 1, 0, vp(MB), 16, 16, vp(MB), 16, 16, vp(MB), 16, 16, vp(MB),
                                        vp(MB), vp(MB), vp(MB), vp(MB), 0, None)

    def size(n=2, nq=40, nk=40):
        return lib.kdn_prompt_attention_workspace_size(n, nq, 1, 1, 64, 1, 0)

    assert call(**{what: MOST}) == 5 and call(**{what: MOST + 1}) == 2 and call(**{what: 2 ** 31 - 1}) == 2
    assert size(**{what: MOST}) > 0 and (size(**{what: MOST + 1}) == 0 or what == "nk")


@pytest.mark.parametrize("what", ["n_free", "cap"])
def test_plan_counts(lib, what):  # noqa: F811
    def call(n_free=20, cap=64):
        return lib.kdn_cache_plan(4, 16, 8, n_free, cap, *[vp(MB)] * 12, 0, None)

    assert call(**{what: MOST}) == 5 and call(**{what: MOST + 1}) == 2 and call(**{what: 2 ** 31 - 1}) == 2
