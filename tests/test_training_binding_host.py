"""What the training operators' Python entry points make of views and of
arguments that are not plain numbers.  Runs without a GPU: each call returns
before it reaches the library."""
import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q


def act(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def one_row(n, width, dtype=torch.bfloat16):
    """One row in memory, n in the view."""
    return act(1, width, dtype=dtype).expand(n, width)


@pytest.mark.parametrize("call", [
    lambda: Q.ln_args(one_row(4, 64)),
    lambda: Q.ln_args(act(0, 64), one_row(3, 64)),
    lambda: Q.ln_args(act(0, 64), None, one_row(3, 64, torch.float32)),
    lambda: Q.grad_args(head_dim=64, dq=one_row(4, 64), n_heads_q=1, tokens=4),
    lambda: Q.grad_args(head_dim=64, dv=one_row(4, 64), n_heads_v=1, tokens=4),
    lambda: Q.attn_args(one_row(4, 64), act(0, 64), act(0, 64), 1, 1, 64),
    lambda: Q.attn_args(act(0, 64), one_row(4, 64), act(4, 64), 1, 1, 64),
    lambda: Q.attn_args(act(0, 64), act(0, 64), one_row(4, 64), 1, 1, 64),
    # the operators that were there before take rows the same way
    lambda: Q.make_args(head_dim=64, q=one_row(4, 64), n_heads_q=1),
    lambda: Q.adaln_args(one_row(4, 64), act(1, 64), act(1, 64)),
])
def test_an_expanded_row_is_refused(built_lib, call):
    # its row stride of 0 would read as the library's default: rows behind the only one
    with pytest.raises(ValueError, match="expanded"):
        call()


def test_one_row_expanded_to_one_is_a_row():
    with pytest.raises(ValueError, match="CUDA"):
        Q._rows(one_row(1, 64), "x")


@pytest.fixture
def calls(built_lib, monkeypatch):
    """The argument structs that reach the library, without a device."""
    seen = []
    Q.load()
    monkeypatch.setattr(Q, "_plans", {})
    monkeypatch.setattr(Q, "_call", lambda fn, a, stream, like: seen.append(a))
    monkeypatch.setattr(Q, "_empty", lambda shape, dtype, like, stream: torch.empty(shape, dtype=dtype))
    return seen


def test_a_number_in_a_tensor_is_read_at_every_call(calls):
    # the tensor is the same object, its value is not
    number = torch.tensor(0.5)
    for value in (0.5, 2.0, 0.25):
        number.fill_(value)
        Q.attention(act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, scale=number, status=False)
        assert calls[-1].scale == value
        Q.layer_norm(act(0, 64), eps=number, status=False, mean=None, rstd=None)
        assert calls[-1].eps == value
    assert not Q._plans


def test_plain_numbers_share_a_plan(calls):
    for _ in range(3):
        Q.attention(act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, scale=0.5, causal=True, status=False)
    assert len(Q._plans) == 1 and all(a.scale == 0.5 and a.causal == 1 for a in calls)
