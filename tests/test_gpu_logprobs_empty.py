"""Log probabilities of no rows, which a filter of answers may leave: nothing to do, where some would be taken."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_rows(gpt_lib, dtype):
    from decoder_only_transformer_gpt_gb300 import binding
    z = torch.randn(5, 300, device="cuda").to(dtype)
    none = z[torch.zeros(5, dtype=torch.bool, device="cuda")]
    for x in (none, z[:0], z[3:3, :200]):
        V = x.shape[1]
        t, row, stats = empty(0, dtype=torch.int32), empty(0), empty(0, 2)
        binding.logprobs(x, t, row, entropy=row, stats=stats, top_ids=empty(0, 4, dtype=torch.int32), top_logp=empty(0, 4))
        binding.logprobs(x, None, None, entropy=row)
        binding.logprobs_bwd(x, t, stats, row, empty(0, V, dtype=dtype), row, row)
        binding.logprobs_bwd(x, t, stats, row, x)
        binding.logprobs_bwd(x, None, stats, None, x, row, row)
    binding.status()


def test_what_some_rows_would_not_be_taken_with_none_are_not(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    x, t, row, stats = empty(0, 20), empty(0, dtype=torch.int32), empty(0), empty(0, 2)
    for call in (lambda: binding.logprobs(x, t, None), lambda: binding.logprobs(x, None, None),
                 lambda: binding.logprobs(x, t, row, top_ids=empty(0, 4, dtype=torch.int32)),
                 lambda: binding.logprobs(x, t, row, top_ids=empty(0, 21, dtype=torch.int32), top_logp=empty(0, 21)),
                 lambda: binding.logprobs(empty(0, 0), t, row),
                 lambda: binding.logprobs_bwd(x, t, stats, None, x), lambda: binding.logprobs_bwd(x, None, stats, None, x),
                 lambda: binding.logprobs_bwd(x, t, stats, row, x, row)):
        with pytest.raises(binding.GptError) as e:
            call()
        assert e.value.code == binding.GPT_EINVAL
    for call in (lambda: binding.logprobs(x, t, empty(1)), lambda: binding.logprobs_bwd(x, t, stats, row, empty(0, 19))):
        with pytest.raises(ValueError):
            call()
