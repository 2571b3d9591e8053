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


def test_tokens_begin_at_any_element(N, R):
    """The library takes token numbers on 16 bytes: slices that begin elsewhere are copied, others passed on as they are."""
    s = R.TokenScorer(6, 100, 4, device="cpu")
    z, tokens = torch.zeros(7, 100), torch.arange(8, dtype=torch.int32)
    base = tokens.data_ptr()
    assert base % 16 == 0
    for n, first in ((6, 0), (6, 1), (3, 2), (4, 4), (1, 7)):
        s.score(z[:n], tokens[first:first + n], stream=7)
        at = R.recorder.calls[-1][1][5]
        assert at % 16 == 0 and (at == base + 4 * first) == (first % 4 == 0)
        if first % 4:
            assert torch.equal(s._shifted[:n], tokens[first:first + n]) and at == s._shifted.data_ptr()


@pytest.mark.parametrize("Hk,Hv,dk,dv", [(1, 1, 32, 32), (16, 48, 128, 128), (128, 128, 128, 128), (64, 512, 128, 128), (1000, 1000, 128, 128),
                                         (2048, 2048, 32, 32), (1, 4096, 64, 128)])
def test_prompts_workspace_has_a_bound(N, Hk, Hv, dk, dv):
    """1000 MiB, however many heads fit two chunks into them; the two chunks where none do."""
    assert 0 < N.gdn_prefill_workspace_bytes(dims(N, Hk=Hk, Hv=Hv, dk=dk, dv=dv)) <= 1000 << 20
    many = N.gdn_prefill_workspace_bytes(dims(N, Hk=16384, Hv=16384, dk=128, dv=128))
    assert many == 2 * 16384 * (4 * 64 * 128 * 2 + 2 * 64 * 64 * 4 + 2 * 128 * 64 * 2 + 64 * 128 * 4 + 144 * 4)
