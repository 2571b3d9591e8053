"""What the prompt, single-token and log-probability calls accept and pass on, beside test_sequences_host.py (no GPU)."""
import pytest
import torch

from test_sequences_host import P, N, R, Recorder, banks, both, dims, status, tensors  # noqa: F401


@pytest.mark.parametrize("dtype,at,fine", [(0, 4, True), (0, 12, True), (0, 2, False), (1, 2, True), (1, 14, True), (1, 1, False)])
def test_logits_begin_at_any_element(N, dtype, at, fine):
    """Of a call whose err is NULL: what is refused is that, or the logits before it."""
    with pytest.raises(N.GdnError) as e:
        N.gdn_top_logprobs(4, 1000, 1000, dtype, P + at, None, 4, P, P, None, P, None, 0)
    assert e.value.status == N.GDN_ERR_INVALID_ARG
    assert ("err" if fine else "logits") in str(e.value)
