"""Sliding-window attention's argument checks, without a GPU (the pointers are never dereferenced)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    from decoder_only_transformer_gpt_gb300 import binding, build
    build.build()
    return binding.load()


def _fwd(lib, **k):
    a = dict(qkv=P, y=P, lse2=P, B=2, T=100, H=4, Hkv=2, D=64, window=16, sinks=4)
    a.update(k)
    return lib.gptk_attention_window(*a.values(), None)


def _bwd(lib, **k):
    a = dict(qkv=P, y=P, dy=P, lse2=P, dqkv=P, B=2, T=100, H=4, Hkv=2, D=64, window=16, sinks=4)
    a.update(k)
    return lib.gptk_attention_window_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_arguments(lib, call):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (dict(qkv=None), dict(y=None), dict(B=0), dict(T=0), dict(H=0), dict(Hkv=0), dict(D=0), dict(window=0),
                dict(window=-3), dict(sinks=-1), dict(T=1 << 30), dict(B=1 << 20, T=1 << 20), dict(H=1 << 26, Hkv=1)):
        assert call(lib, **bad) == binding.GPT_EINVAL, bad
    for bad in (dict(D=48), dict(D=128), dict(H=3), dict(qkv=ODD), dict(y=ODD)):
        assert call(lib, **bad) == binding.GPT_ECONFIG, bad


def test_derivative_pointers(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    for name in ("dy", "lse2", "dqkv"):
        assert _bwd(lib, **{name: None}) == binding.GPT_EINVAL
    for name in ("dy", "dqkv"):
        assert _bwd(lib, **{name: ODD}) == binding.GPT_ECONFIG


@pytest.mark.parametrize("bad", ["dtype", "width", "strides", "device", "lse2"])
def test_binding_refuses_tensors(lib, bad):
    from decoder_only_transformer_gpt_gb300 import binding
    qkv, y, lse2 = (torch.zeros(2, 50, 8 * 32, dtype=torch.bfloat16), torch.zeros(2, 50, 4 * 32, dtype=torch.bfloat16),
                    torch.zeros(2, 4, 50))
    if bad == "dtype":
        qkv = qkv.float()
    elif bad == "width":
        qkv = torch.zeros(2, 50, 8 * 32 + 1, dtype=torch.bfloat16)
    elif bad == "strides":
        qkv = qkv.transpose(0, 1)
    elif bad == "lse2":
        lse2 = lse2.double()
    with pytest.raises(ValueError):
        binding.attention_window(qkv, y, 4, 2, 8, 1, lse2=lse2)
    with pytest.raises(ValueError):
        binding.attention_window_bwd(qkv, y, y, lse2, qkv, 4, 2, 8, 1)


def test_reference_gradient_against_differences():
    # the plain derivative that the GPU tests use, against central differences of the plain forward
    import numpy as np

    import window_ref
    rng = np.random.default_rng(0)
    for T, W, S in ((7, 3, 2), (6, 1, 0), (5, 9, 0), (8, 2, 8)):
        q, k, u, dy = (rng.standard_normal((T, 4)) for _ in range(4))
        got = window_ref.backward(q, k, u, dy, W, S)
        for which, x in enumerate((q, k, u)):
            for i in np.ndindex(*x.shape):
                args, h = [q, k, u], 1e-5
                args[which] = x.copy()
                args[which][i] += h
                up = (window_ref.forward(*args, W, S)[0] * dy).sum()
                args[which][i] -= 2 * h
                down = (window_ref.forward(*args, W, S)[0] * dy).sum()
                assert abs((up - down) / (2 * h) - got[which][i]) < 1e-8 * (1 + abs(got[which][i])) / h * 1e-5 + 1e-7
