"""A workspace of the log probabilities holds every smaller call, without a GPU."""

import pytest

import zero_sharded_mixed_step_gb300 as zs


@pytest.mark.parametrize("vocab,width", [(1, 8), (7, 8), (17, 16), (255, 64), (257, 64), (5000, 128), (50257, 768)])
@pytest.mark.parametrize("with_grad", [False, True])
def test_every_smaller_call_fits(zlib, vocab, width, with_grad):
    tops = [k for k in (0, 1, 8, 9, 16) if k <= vocab]
    counts = [0, 1, 31, 32, 33, 95, 96, 97, 127, 128, 129, 255, 256, 257, 1000, 32768, 32768 + 100, 70_000]
    for k, tokens in enumerate(counts):
        for j, top in enumerate(tops):
            whole = zs.zero_lm_logprobs_workspace_bytes(tokens, vocab, width, top, with_grad)
            for fewer in counts[:k + 1]:
                for less in tops[:j + 1]:
                    assert zs.zero_lm_logprobs_workspace_bytes(fewer, vocab, width, less, with_grad) <= whole
