"""Arguments of the attention calls that are not what they should be are refused by name, on the host."""
import pytest
import torch

from selective_state_space_prefill_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    build.build_calls()


class NoTruth:
    def __bool__(self):
        raise RuntimeError("neither")


@pytest.mark.parametrize("value", [NoTruth(), torch.zeros(2)])
def test_interleaved_must_have_a_truth_value(value):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache, i32 = torch.zeros(2, 2, 16, 64, dtype=torch.int8), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="interleaved"):
        binding.attn_append(None, x, x, None, None, None, cache, cache, i32, interleaved=value)
