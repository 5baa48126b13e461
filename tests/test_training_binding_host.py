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


class Elsewhere:
    """What the binding asks of a CUDA tensor, without a device."""
    is_cuda = True

    def __init__(self, device, *shape, dtype=torch.bfloat16, like=None):
        self.like = torch.empty(*shape, dtype=dtype, device="meta") if like is None else like
        self.device, self.shape, self.dtype = torch.device("cuda", device), self.like.shape, self.like.dtype

    def __getattr__(self, name):
        return getattr(self.like, name)

    def __getitem__(self, at):
        return Elsewhere(self.device.index, like=self.like[at])

    def view(self, *shape):
        return Elsewhere(self.device.index, like=self.like.view(*shape))

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 0


def rows(device):
    return Elsewhere(device, 4, 128)


def vector(device, n=4):
    return Elsewhere(device, n, dtype=torch.float32)


def ints(device, n=1):
    return Elsewhere(device, n, dtype=torch.int32)


def table(device):
    return Elsewhere(device, 4, 128, dtype=torch.float32)


def packed(device):
    return Elsewhere(device, 4, 384)


@pytest.mark.parametrize("call", [
    lambda: Q.layer_norm(rows(0), vector(1, 128)),
    lambda: Q.layer_norm(rows(0), None, vector(1, 128)),
    lambda: Q.layer_norm(rows(0), out=rows(1)),
    lambda: Q.layer_norm(rows(0), mean=vector(1)),
    lambda: Q.layer_norm(rows(0), rstd=vector(1)),
    lambda: Q.layer_norm(rows(0), dev_status=ints(1)),
    lambda: Q.layer_norm_backward(rows(1), rows(0), None, vector(0), vector(0)),
    lambda: Q.layer_norm_backward(rows(0), rows(0), None, vector(0), vector(1)),
    lambda: Q.layer_norm_backward(rows(0), rows(0), None, vector(0), vector(0), dweight=vector(1, 128)),
    lambda: Q.layer_norm_backward(rows(0), rows(0), None, vector(0), vector(0), status=False, workspace=vector(1, 1 << 20)),
    lambda: Q.qk_norm_rope_packed_backward(packed(1), packed(0), 1, 1, 1, 128, vector(0, 128), vector(0, 128), table(0), table(0)),
    lambda: Q.qk_norm_rope_packed_backward(packed(0), packed(0), 1, 1, 1, 128, vector(0, 128), vector(1, 128),
                                           table(0), table(0)),
    lambda: Q.qk_norm_rope_packed_backward(packed(0), packed(0), 1, 1, 1, 128, vector(0, 128), vector(0, 128),
                                           table(0), table(1)),
    lambda: Q.attention(rows(0), rows(1), rows(0), 1, 1, 128),
    lambda: Q.attention(rows(0), rows(0), rows(1), 1, 1, 128),
    lambda: Q.attention(rows(0), rows(0), rows(0), 1, 1, 128, k_lens=ints(1)),
    lambda: Q.attention(rows(0), rows(0), rows(0), 1, 1, 128, lse=vector(1)),
    lambda: Q.attention_backward(rows(0), rows(0), rows(0), rows(0), rows(1), vector(0), 1, 1, 128),
    lambda: Q.attention_backward(rows(0), rows(0), rows(0), rows(0), rows(0), vector(0), 1, 1, 128, dv=rows(1)),
])
def test_tensors_of_two_devices_are_refused(calls, call):
    with pytest.raises(ValueError, match="device"):
        call()
    assert not calls


def test_a_call_runs_on_its_tensors_device(built_lib, monkeypatch):
    # the library launches on the calling thread's device: it has to be the tensors'
    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Stream:
        def __init__(self, device):
            self.device_index, self.cuda_stream = device, 7

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)

    def fn(a, s):
        seen.append((current[0], s))
        return 0

    for device in (0, 1):
        Q._call(fn, Q.QknrAttnArgs(), None, rows(device))
        Q._call(fn, Q.QknrAttnArgs(), Stream(device), rows(device))
    assert seen == [(0, 100), (0, 7), (1, 101), (1, 7)] and current == [0]
    with pytest.raises(ValueError, match="device"):
        Q._call(fn, Q.QknrAttnArgs(), Stream(1), rows(0))
    assert len(seen) == 4


@pytest.mark.parametrize("stride", [1, 7, 129, 131])
def test_the_stride_of_a_single_row_says_nothing(calls, stride):
    # tensors of one row have whatever row stride they were made with
    row = Elsewhere(0, like=torch.empty(1000, dtype=torch.bfloat16, device="meta").as_strided((1, 128), (stride, 1)))
    Q.attention(row, row, row, 1, 1, 128, status=False)
    assert (calls[-1].q_stride, calls[-1].k_stride, calls[-1].v_stride) == (0, 0, 0)
    Q.layer_norm(row, None, None, out=row, status=False)
    assert (calls[-1].x_stride, calls[-1].y_stride) == (0, 0)
