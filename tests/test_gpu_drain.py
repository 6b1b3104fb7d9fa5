"""A kernel that gave up a wait stays until its copies in flight have landed."""

import pytest

from grouped_query_attention_attn_b200 import _binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("us", [500, 20000, 200000])
def test_drain_outlasts_the_abort(gqa_lib, us):
    # what is in flight lands us / 2 after the wait gave up; GQA_ERR_CUDA: it was not waited for
    assert _binding.gqa_selftest_wait_timeout(us) == _binding.GQA_ERR_TIMEOUT
    assert _binding.gqa_device_status(0) == _binding.GQA_OK
