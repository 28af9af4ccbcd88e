"""What the Python calls of the 4-bit cache refuse before the library sees it.  CPU only."""
import shutil

import pytest
import torch


@pytest.fixture(scope="module")
def pa():
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not available")
    import paged_kv_cache_09_gb300
    paged_kv_cache_09_gb300.build()
    return paged_kv_cache_09_gb300


PAST = 2**32  # a C int of this is 0


def test_lengths_past_32_bits_are_refused(pa):
    # (They came to the library without their upper bits.)
    with pytest.raises(ValueError):
        pa.prefill_varlen_q4_workspace_size([0, 10], [PAST + 10], True, 24, 4, 256, 832)
    with pytest.raises(ValueError):
        pa.prefill_varlen_q4_workspace_size([0, PAST + 10], [10], True, 24, 4, 256, 832)
    with pytest.raises(ValueError):
        pa.prefill_q4_workspace_size(10, PAST, True, 24, 4, 256, 832)
    with pytest.raises(ValueError):
        pa.prefill_q4_workspace_size(PAST + 10, 0, True, 24, 4, 256, 832)
    with pytest.raises(ValueError):
        pa.decode_q4_workspace_size(1, 24, 4, 256, 832, PAST + 100)
    with pytest.raises(ValueError):
        pa.batch_input_prep(None, None, [None], [16], [None], PAST)


def test_prefill_chunk_refuses_what_is_no_cuda_tensor(pa):
    q = torch.zeros(3, 6, 256, dtype=torch.bfloat16)
    cache = torch.zeros(pa.q4_cache_shape(1, 16, 1), dtype=torch.uint8)
    table = torch.zeros(1, dtype=torch.int32)
    for args in ((None, table), (q, [0]), (q, table)):
        with pytest.raises(TypeError):
            pa.prefill_chunk_q4(args[0], cache, cache, args[1], 0, True, 0.0625)
