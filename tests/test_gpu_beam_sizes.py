"""Selections of more tokens than 32 bits count."""

import pytest

pytestmark = pytest.mark.gpu


def test_more_tokens_than_32_bits_count_are_refused():
    import torch

    import affine_bit_matmul_gb300 as mxq

    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 9 GB")
    logits = torch.empty((1, 2 ** 32 + 5), dtype=torch.bfloat16, device="cuda")
    logits[0, :5] = torch.arange(5)
    scores = torch.zeros((1, 1), device="cuda")
    for kw in ({}, dict(stream=torch.cuda.current_stream())):
        with pytest.raises(mxq.MxqError) as e:
            mxq.beam_select(logits, scores, **kw)
        assert e.value.status == 3
    # rows that lie as far apart
    ends = logits.as_strided((2, 5), (2 ** 32, 1))
    ends.copy_(torch.tensor([[0.0, 1, 2, 3, 4], [0, 5, 0, 0, 0]]))
    got = mxq.beam_select(ends, torch.zeros((1, 2), device="cuda"))
    assert got[1].tolist() == [[1, 0]] and got[2].tolist() == [[1, 4]]
    del ends, logits
    torch.cuda.empty_cache()
