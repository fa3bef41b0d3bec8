"""Sizes of a prompt's workspace that a 32-bit field does not hold, without a GPU."""
import pytest

from mla_attention_decode_gb300 import binding, build, prompt


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("by", [1 << 32, -(1 << 32), 1 << 31])
@pytest.mark.parametrize("place", range(4))
def test_sizes_that_would_wrap_are_refused(place, by):
    sizes = [5, 10, 1, 16]
    sizes[place] += by
    with pytest.raises(binding.MLAError) as e:
        prompt.MLAPrompt(*sizes, device="cpu")
    assert e.value.status == binding.MLA_ERR_INVALID_ARG
