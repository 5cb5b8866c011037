"""The C entry point of differential attention's backward where there is nothing to add up: dlambda is zero."""
import ctypes

import pytest
import torch

import ulysses_dit_attention_gb300 as uaa

P = ctypes.c_void_p


def _bwd(dlam, B, Sq, Sk, H=3, dtype=2, stream=None):
    f = P(1 << 20)  # tensors without an element: never read
    return uaa.lib().uaa_diff_attn_bwd(f, f, f, f, dtype, f, f, f, f, None, f, f, f, dlam, B, Sq, Sk, H, 64,
                                       ctypes.c_float(0.1), None, 0, stream)


def test_refusals():
    err = lambda: uaa.lib().uaa_last_error().decode()  # noqa: E731
    assert _bwd(None, 0, 4, 5) == -1 and "lambda" in err()
    assert _bwd(P((1 << 20) + 2), 2, 0, 0) == -1 and "aligned" in err()
    assert _bwd(P(1 << 20), 0, 4, 5, dtype=1) == -1
    assert _bwd(None, 0, 4, 5, H=0) == 0 and _bwd(None, 2, 4, 5, H=0) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,Sq,Sk", [(0, 4, 5), (2, 0, 0), (0, 0, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dlambda_is_written(B, Sq, Sk, dtype):
    dlam = torch.full((5,), 7.0, dtype=dtype, device="cuda")
    st = _bwd(P(dlam[:3].data_ptr()), B, Sq, Sk, dtype=0 if dtype == torch.bfloat16 else 2,
              stream=P(torch.cuda.current_stream().cuda_stream))
    assert st == 0 and dlam.tolist() == [0.0, 0.0, 0.0, 7.0, 7.0]
