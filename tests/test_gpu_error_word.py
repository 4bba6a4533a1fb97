"""fa_check_device_error reports every kind of error that was met since it was
last asked, one to a call: neither kind hides the other."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


@pytest.mark.parametrize("index_first", [True, False])
def test_a_wait_that_ran_out_and_a_bad_index(fa, index_first):
    q, k, v = (torch.randn(1, 2, 512, 64, device="cuda").bfloat16() for _ in range(3))
    pages = torch.zeros((4, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream

    def bad_index():  # a page that the cache does not have
        fa.cache_append(pages[0, :, :1].transpose(0, 1).contiguous(), pages[1, :, :1].transpose(0, 1).contiguous(), pages, pages.clone(), ints([[9]]), ints([0, 1]), ints([1]))

    def timeout():
        assert fa.lib().fa_debug_inject(1) == fa.FA_OK
        fa.fwd_window(q, k, v, 512)

    fa.check_device_error()
    for call in (bad_index, timeout) if index_first else (timeout, bad_index):
        call()
    found = [fa.lib().fa_check_device_error(stream) for _ in range(3)]
    assert found == [fa.FA_ERR_TIMEOUT, fa.FA_ERR_INDEX, fa.FA_OK]
