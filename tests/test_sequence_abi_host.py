"""What the C entry points of the RMS norm, of attention over packed sequences
and beside a shared prefix refuse, each before any CUDA call, and what their
binding refuses.  Runs without a GPU: addresses are plain integers that are
never touched."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from diffusion_transformer_qk_gb300 import build as B
from diffusion_transformer_qk_gb300 import qknr as Q
from tests.test_training_abi_host import (ABI, ALIGN, FAKE, INCLUDE, NULL, OVERLAP, SHAPE, STEP, UNSUPPORTED, act, changed, fake,
                                          lib, refused)  # noqa: F401  (lib: the fixture)
from tests.test_training_binding_host import calls, ints, one_row, rows, vector  # noqa: F401  (calls: the fixture)

host = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only tests with fake device addresses")
pytestmark = host


def rms(T=600, C=1536, small=False):
    a = Q.QknrRmsArgs()
    Q.load().qknr_rms_args_init(ctypes.byref(a))
    a.x, a.residual, a.sum, a.y, a.weight, a.rstd, a.scales, a.dy, a.dsum, a.dx, a.dweight, a.workspace = (fake(i) for i in range(12))
    a.workspace_bytes, a.tokens, a.hidden = STEP, T, C
    if small:
        a.out = Q.RMS_OUT_E4M3
    return a


def pack(Hq=6, Hk=2, D=64):
    a = Q.QknrPackArgs()
    Q.load().qknr_pack_args_init(ctypes.byref(a))
    (a.q, a.k, a.v, a.o, a.lse, a.q_starts, a.k_starts, a.dout, a.dq, a.dk, a.dv, a.workspace) = (fake(i) for i in range(12))
    a.workspace_bytes, a.batch, a.rows_q, a.rows_k = STEP, 5, 7000, 9000     # long enough to need a workspace
    a.n_heads_q, a.n_heads_k, a.head_dim = Hq, Hk, D
    return a


def prefix(Hq=6, Hk=2, D=64):
    a = Q.QknrPrefixArgs()
    Q.load().qknr_prefix_args_init(ctypes.byref(a))
    (a.q, a.k, a.v, a.prefix_k, a.prefix_v, a.o, a.lse, a.q_lens, a.k_lens, a.workspace) = (fake(i) for i in range(10))
    a.workspace_bytes, a.batch, a.seq_q, a.seq_k, a.prefix = STEP, 64, 1, 100, 4000
    a.n_heads_q, a.n_heads_k, a.head_dim = Hq, Hk, D
    return a


def test_struct_layouts_match(lib):  # noqa: F811
    assert lib.qknr_rms_sizeof_args() == ctypes.sizeof(Q.QknrRmsArgs)
    assert lib.qknr_pack_sizeof_args() == ctypes.sizeof(Q.QknrPackArgs)
    assert lib.qknr_prefix_sizeof_args() == ctypes.sizeof(Q.QknrPrefixArgs)


@pytest.mark.parametrize("struct,init,defaults", [
    ("QknrRmsArgs", "qknr_rms_args_init", dict(dtype=Q.BF16, param_dtype=Q.FP32)),
    ("QknrPackArgs", "qknr_pack_args_init", dict(dtype=Q.BF16)),
    ("QknrPrefixArgs", "qknr_prefix_args_init", dict(dtype=Q.BF16)),
])
def test_init_writes_every_field(lib, struct, init, defaults):  # noqa: F811
    a = getattr(Q, struct)()
    ctypes.memset(ctypes.byref(a), 0xFF, ctypes.sizeof(a))
    getattr(lib, init)(ctypes.byref(a))
    getattr(lib, init)(None)
    assert a.abi_version == Q.ABI_VERSION
    eps = getattr(a, "eps", None)
    assert eps is None or abs(eps - 1e-6) < 1e-12
    for name, _ in a._fields_:
        if name not in ("abi_version", "eps"):
            assert getattr(a, name) in (defaults.get(name, 0), None), name


@pytest.mark.parametrize("fn", ["qknr_rms_forward", "qknr_rms_backward", "qknr_pack_forward", "qknr_pack_backward",
                                "qknr_prefix_forward"])
def test_null_args(lib, fn):  # noqa: F811
    assert getattr(lib, fn)(None, None) == NULL


@pytest.mark.parametrize("fn,make", [("qknr_rms_workspace_bytes", rms), ("qknr_pack_workspace_bytes", pack),
                                     ("qknr_pack_backward_workspace_bytes", pack), ("qknr_prefix_workspace_bytes", prefix)])
def test_workspace_queries(lib, fn, make):  # noqa: F811
    n = ctypes.c_size_t(7)
    assert getattr(lib, fn)(None, ctypes.byref(n)) == NULL and n.value == 0
    assert getattr(lib, fn)(ctypes.byref(make()), None) == NULL
    assert getattr(lib, fn)(ctypes.byref(make()), ctypes.byref(n)) == 0 and n.value > 0
    a = changed(make, dict(dtype=9))
    assert getattr(lib, fn)(ctypes.byref(a), ctypes.byref(n)) == UNSUPPORTED and n.value == 0


RMS_BOTH = [
    (dict(abi_version=99), ABI), (dict(dtype=Q.FP32), UNSUPPORTED), (dict(param_dtype=Q.FP16), UNSUPPORTED),
    (dict(hidden=0), UNSUPPORTED), (dict(hidden=1540), UNSUPPORTED), (dict(hidden=32776), UNSUPPORTED),
    (dict(tokens=-1), SHAPE), (dict(rows_per_batch=-1), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(out=2), UNSUPPORTED), (dict(scale_block=64), UNSUPPORTED), (dict(scale_block=128), UNSUPPORTED),
    (dict(x=None), NULL), (dict(x_stride=1528), SHAPE), (dict(param_stride=8), SHAPE), (dict(x_stride=1540), ALIGN),
    (dict(x=FAKE + 8), ALIGN), (dict(weight=fake(4) + 4), ALIGN), (dict(param_stride=1538), ALIGN), (dict(rstd=fake(5) + 1), ALIGN),
]


@pytest.mark.parametrize("change,expect", RMS_BOTH + [
    (dict(y=None), NULL), (dict(sum=None), NULL), (dict(residual_stride=1528), SHAPE), (dict(sum_stride=1540), ALIGN),
    (dict(residual=fake(1) + 2), ALIGN), (dict(y=fake(3) + 8), ALIGN), (dict(y_stride=8), SHAPE),
    (dict(y=FAKE + 16), OVERLAP), (dict(y=FAKE, y_stride=1544), OVERLAP), (dict(y=fake(1)), OVERLAP), (dict(y=fake(2)), OVERLAP),
    (dict(sum=FAKE + 16), OVERLAP), (dict(sum=fake(1), sum_stride=1544), OVERLAP), (dict(sum=fake(4)), OVERLAP),
    (dict(y=fake(4)), OVERLAP), (dict(y=fake(5)), OVERLAP), (dict(rstd=FAKE), OVERLAP), (dict(rstd=fake(1) + 64), OVERLAP),
    (dict(rstd=fake(2)), OVERLAP), (dict(rstd=fake(4)), OVERLAP),
])
def test_rms_norm_refuses(lib, change, expect):  # noqa: F811
    refused(lib, "qknr_rms_forward", changed(rms, change), expect)


@pytest.mark.parametrize("change,expect", [
    (dict(scales=None), NULL), (dict(scales=fake(6) + 2), ALIGN), (dict(scale_block=128, hidden=1544), UNSUPPORTED),
    (dict(y=fake(3) + 4), ALIGN), (dict(y_stride=1540), ALIGN), (dict(y=FAKE), OVERLAP), (dict(y=fake(1) + 8), OVERLAP),
    (dict(scales=FAKE), OVERLAP), (dict(scales=fake(3)), OVERLAP), (dict(scales=fake(5) + 599 * 4), OVERLAP),
    (dict(scales=fake(5) - 600 * 12 * 4 + 4, scale_block=128), OVERLAP), (dict(scales=fake(2)), OVERLAP),
])
def test_quantized_rms_norm_refuses(lib, change, expect):  # noqa: F811
    refused(lib, "qknr_rms_forward", changed(lambda: rms(small=True), change), expect)


@pytest.mark.parametrize("change,expect", RMS_BOTH + [
    (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(rstd=None), NULL), (dict(workspace=None), NULL),
    (dict(workspace_bytes=16), SHAPE), (dict(workspace=fake(11) + 8), ALIGN), (dict(dweight=fake(10) + 4), ALIGN),
    (dict(dsum_stride=1528), SHAPE), (dict(dsum=fake(8) + 2), ALIGN), (dict(dx_stride=1540), ALIGN),
    (dict(dx=FAKE), OVERLAP), (dict(dx=fake(7) + 16), OVERLAP), (dict(dx=fake(8), dx_stride=1544), OVERLAP),
    (dict(dx=fake(4)), OVERLAP), (dict(dx=fake(5)), OVERLAP), (dict(dx=fake(10)), OVERLAP), (dict(dweight=fake(7)), OVERLAP),
    (dict(dweight=FAKE), OVERLAP), (dict(workspace=fake(8)), OVERLAP), (dict(workspace=fake(10)), OVERLAP),
])
def test_rms_norm_backward_refuses(lib, change, expect):  # noqa: F811
    refused(lib, "qknr_rms_backward", changed(rms, change), expect)


ATTN = [
    (dict(abi_version=9), ABI), (dict(dtype=Q.FP32), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(n_heads_q=5), SHAPE),
    (dict(n_heads_k=0), SHAPE), (dict(batch=-1), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(lse=None), NULL),
    (dict(q=FAKE + 8), ALIGN), (dict(v_stride=132), ALIGN), (dict(k_stride=64), SHAPE), (dict(lse=fake(3) + 2), ALIGN),
    (dict(workspace=None), NULL), (dict(workspace_bytes=64), SHAPE), (dict(o_stride=1 << 31), UNSUPPORTED),
]


@pytest.mark.parametrize("change,expect", ATTN + [
    (dict(rows_q=-1), SHAPE), (dict(rows_k=-1), SHAPE), (dict(q_starts=None), NULL), (dict(q_starts=fake(5) + 2), ALIGN),
    (dict(k_starts=fake(6) + 1), ALIGN), (dict(o=None), NULL), (dict(o=FAKE), OVERLAP), (dict(o=fake(1)), OVERLAP),
    (dict(o=fake(4)), OVERLAP), (dict(o=fake(5)), OVERLAP), (dict(lse=fake(6)), OVERLAP), (dict(lse=fake(11)), OVERLAP),
    (dict(workspace=fake(2)), OVERLAP), (dict(workspace=fake(5)), OVERLAP), (dict(o=fake(11) + 64), OVERLAP),
    (dict(workspace=fake(11) + 8), ALIGN), (dict(rows_q=0x7fffffff), UNSUPPORTED), (dict(batch=0x7fffffff), UNSUPPORTED),
])
def test_packed_attention_refuses(lib, change, expect):  # noqa: F811
    refused(lib, "qknr_pack_forward", changed(pack, change), expect)


@pytest.mark.parametrize("change,expect", ATTN + [
    (dict(q_starts=None), NULL), (dict(dout=None), NULL), (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dv=None), NULL),
    (dict(dq=FAKE), OVERLAP), (dict(dk=fake(2)), OVERLAP), (dict(dv=fake(7)), OVERLAP), (dict(dq=fake(9)), OVERLAP),
    (dict(dk=fake(4)), OVERLAP), (dict(dv=fake(5)), OVERLAP), (dict(workspace=fake(3)), OVERLAP), (dict(workspace=fake(6)), OVERLAP),
    (dict(dk=fake(9), dv=fake(9) + 64), OVERLAP), (dict(dout_stride=8), SHAPE), (dict(dq_stride=388), ALIGN),
])
def test_packed_attention_backward_refuses(lib, change, expect):  # noqa: F811
    refused(lib, "qknr_pack_backward", changed(pack, change), expect)


@pytest.mark.parametrize("change,expect", ATTN[:-1] + [
    (dict(seq_q=-1), SHAPE), (dict(prefix=-1), SHAPE), (dict(prefix_k=None), NULL), (dict(prefix_v=None), NULL),
    (dict(prefix_k=fake(3) + 8), ALIGN), (dict(prefix_v_stride=132), ALIGN), (dict(prefix_k_stride=64), SHAPE),
    (dict(q_lens=fake(7) + 2), ALIGN), (dict(k_lens=fake(8) + 2), ALIGN), (dict(o=FAKE), OVERLAP), (dict(o=fake(3)), OVERLAP),
    (dict(o=fake(4) + 128), OVERLAP), (dict(o=fake(6)), OVERLAP), (dict(lse=fake(4)), OVERLAP), (dict(lse=fake(7)), OVERLAP),
    (dict(workspace=fake(3)), OVERLAP), (dict(workspace=fake(8)), OVERLAP), (dict(workspace=fake(6)), OVERLAP),
    (dict(prefix=0x7fffffff), UNSUPPORTED), (dict(batch=0x7fffffff), UNSUPPORTED),
])
def test_prefix_attention_refuses(lib, change, expect):  # noqa: F811
    refused(lib, "qknr_prefix_forward", changed(prefix, change), expect)


def test_calls_without_work_need_nothing(lib):  # noqa: F811
    a = Q.QknrRmsArgs()
    lib.qknr_rms_args_init(ctypes.byref(a))
    a.hidden = 64
    assert lib.qknr_rms_forward(ctypes.byref(a), None) == 0 and lib.qknr_rms_backward(ctypes.byref(a), None) == 0
    a = Q.QknrPackArgs()
    lib.qknr_pack_args_init(ctypes.byref(a))
    a.head_dim, a.n_heads_q, a.n_heads_k = 64, 4, 2
    assert lib.qknr_pack_forward(ctypes.byref(a), None) == 0 and lib.qknr_pack_backward(ctypes.byref(a), None) == 0
    a.batch, a.q_starts = 3, FAKE
    assert lib.qknr_pack_forward(ctypes.byref(a), None) == 0 and lib.qknr_pack_backward(ctypes.byref(a), None) == 0
    a = Q.QknrPrefixArgs()
    lib.qknr_prefix_args_init(ctypes.byref(a))
    a.head_dim, a.n_heads_q, a.n_heads_k, a.batch = 64, 4, 2, 3
    assert lib.qknr_prefix_forward(ctypes.byref(a), None) == 0


# ---------------------------------------------------------------------------
# the binding

i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("call", [
    lambda: Q.rms_norm(act(4, 64)),                                              # not on a GPU
    lambda: Q.rms_norm(act(4, 64, dtype=torch.float32)),
    lambda: Q.rms_norm(act(2, 4, 64)),
    lambda: Q.rms_norm(act(0, 64), act(32)),
    lambda: Q.rms_norm(act(0, 64), act(64, dtype=torch.float16)),
    lambda: Q.rms_norm(act(0, 64), residual=act(0, 32)),
    lambda: Q.rms_norm(act(0, 64), residual=act(0, 64, dtype=torch.float16)),
    lambda: Q.rms_norm(act(0, 64), sum_out=act(0, 64)),                          # no residual
    lambda: Q.rms_norm(act(0, 64), out=act(0, 64, dtype=torch.float16)),
    lambda: Q.rms_norm_quantized(act(0, 64), out=act(0, 64)),
    lambda: Q.rms_norm_quantized(act(0, 192), block=128),
    lambda: Q.rms_norm_quantized(act(0, 128), block=64),
    lambda: Q.rms_norm_backward(act(0, 64), act(0, 128), None, act(0)),
    lambda: Q.rms_norm_backward(act(0, 64), act(0, 64), None, act(0, dtype=torch.float32), dsum=act(0, 32)),
    lambda: Q.rms_norm_backward(act(0, 64), act(0, 64), None, act(0, dtype=torch.float32), dweight=act(64, dtype=torch.float32)),
    lambda: Q.attention_packed(act(4, 128), act(4, 128), act(4, 128), 1, 1, 128, i32(2)),         # not on a GPU
    lambda: Q.attention_packed(act(0, 128), act(0, 64), act(0, 128), 1, 1, 128, i32(2)),
    lambda: Q.attention_packed(act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, i32(2)),         # starts on the CPU
    lambda: Q.attention_packed(act(0, 128), act(0, 128), act(0, 128, dtype=torch.float16), 1, 1, 128, i32(2)),
    lambda: Q.attention_packed(act(0, 128), act(0, 128), act(3, 128), 1, 1, 128, i32(2)),
    lambda: Q.attention_prefix(act(0, 128), act(0, 128), act(0, 128), act(0, 64), act(0, 128), 1, 1, 128),
    lambda: Q.attention_prefix(act(0, 128), act(0, 128), act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, batch=0),
    lambda: Q.attention_prefix(act(0, 128), act(0, 128), act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, scale=0.0),
    lambda: Q.attention_prefix(act(0, 128), act(0, 128), act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, k_lens=i32(1)),
    # an expanded row
    lambda: Q.rms_args(one_row(4, 64)),
    lambda: Q.rms_args(act(0, 64), one_row(3, 64, torch.float32)),
    lambda: Q.pack_args(one_row(4, 64), act(0, 64), act(0, 64), 1, 1, 64, i32(2)),
    lambda: Q.pack_args(act(0, 64), act(0, 64), one_row(4, 64), 1, 1, 64, i32(2)),
    lambda: Q.prefix_args(act(0, 64), act(0, 64), act(0, 64), one_row(4, 64), act(0, 64), 1, 1, 64),
])
def test_binding_refuses(lib, call):  # noqa: F811
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [
    lambda: Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(0, 0)),                 # not even one start
    lambda: Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(0, 3), ints(0, 2)),
    lambda: Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, vector(0, 3)),
    lambda: Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(0, 3), lse=vector(0, 5)),
    lambda: Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(0, 3), scale=float("nan")),
    lambda: Q.attention_prefix(rows(0), rows(0), rows(0), rows(0), rows(0), 1, 1, 128, batch=3),
    lambda: Q.attention_prefix(rows(0), rows(0), rows(0), rows(0), rows(0), 1, 1, 128, batch=2, k_lens=ints(0, 3)),
    lambda: Q.rms_norm(rows(0), rstd=vector(0, 5)),
    lambda: Q.rms_norm_quantized(rows(0), scales=vector(0, 5)),
])
def test_binding_refuses_lengths_that_do_not_fit(calls, call):  # noqa: F811
    with pytest.raises(ValueError):
        call()
    assert not calls


@pytest.mark.parametrize("call", [
    lambda: Q.rms_norm(rows(0), residual=rows(1)),
    lambda: Q.rms_norm(rows(0), vector(1, 128)),
    lambda: Q.rms_norm(rows(0), out=rows(1)),
    lambda: Q.rms_norm(rows(0), residual=rows(0), sum_out=rows(1)),
    lambda: Q.rms_norm(rows(0), rstd=vector(1)),
    lambda: Q.rms_norm_quantized(rows(0), scales=vector(1)),
    lambda: Q.rms_norm_backward(rows(0), rows(0), None, vector(0), dsum=rows(1)),
    lambda: Q.rms_norm_backward(rows(1), rows(0), None, vector(0)),
    lambda: Q.rms_norm_backward(rows(0), rows(0), None, vector(1)),
    lambda: Q.attention_packed(rows(0), rows(1), rows(0), 1, 1, 128, ints(0, 3)),
    lambda: Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(1, 3)),
    lambda: Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(0, 3), ints(1, 3)),
    lambda: Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(0, 3), lse=vector(1)),
    lambda: Q.attention_packed_backward(rows(0), rows(0), rows(0), rows(0), rows(1), vector(0), 1, 1, 128, ints(0, 3)),
    lambda: Q.attention_packed_backward(rows(0), rows(0), rows(0), rows(0), rows(0), vector(0), 1, 1, 128, ints(0, 3), dk=rows(1)),
    lambda: Q.attention_prefix(rows(0), rows(0), rows(0), rows(1), rows(0), 1, 1, 128),
    lambda: Q.attention_prefix(rows(0), rows(0), rows(0), rows(0), rows(0), 1, 1, 128, k_lens=ints(1)),
])
def test_tensors_of_two_devices_are_refused(calls, call):  # noqa: F811
    with pytest.raises(ValueError, match="device"):
        call()
    assert not calls


def test_a_number_in_a_tensor_is_read_at_every_call(calls):  # noqa: F811
    number = torch.tensor(0.5)
    for value in (0.5, 2.0, 0.25):
        number.fill_(value)
        Q.rms_norm(act(0, 64), eps=number, status=False)
        assert calls[-1].eps == value
        Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(0, 3), scale=number, status=False)
        assert calls[-1].scale == value
    assert not Q._plans


@pytest.mark.parametrize("stride", [1, 7, 129, 131])
def test_the_stride_of_a_single_row_says_nothing(calls, stride):  # noqa: F811
    from tests.test_training_binding_host import Elsewhere

    row = Elsewhere(0, like=torch.empty(1000, dtype=torch.bfloat16, device="meta").as_strided((1, 128), (stride, 1)))
    Q.rms_norm(row, out=row, status=False)
    assert (calls[-1].x_stride, calls[-1].y_stride) == (0, 0)
    Q.attention_packed(row, row, row, 1, 1, 128, ints(0, 2), status=False)
    assert (calls[-1].q_stride, calls[-1].k_stride, calls[-1].v_stride) == (0, 0, 0)


def test_plans_of_equal_metadata_are_shared_and_others_are_not(calls):  # noqa: F811
    for _ in range(3):
        Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(0, 3), status=False)
    assert len(Q._plans) == 1
    Q.attention_packed(rows(0), rows(0), rows(0), 1, 1, 128, ints(0, 4), status=False)
    assert len(Q._plans) == 2 and calls[-1].batch == 3


# ---------------------------------------------------------------------------
# C

PROGRAM = r"""
#include <stdio.h>
#include "qknr_rms.h"
#include "qknr_pack.h"
#include "qknr_prefix.h"

#define CHECK(cond, code) do { if (!(cond)) { fprintf(stderr, "failed: %s\n", #cond); return code; } } while (0)

int main(void) {
  qknr_rms_args n;
  qknr_pack_args p;
  qknr_prefix_args f;
  size_t bytes = 0;
  CHECK(qknr_rms_sizeof_args() == sizeof n && qknr_pack_sizeof_args() == sizeof p && qknr_prefix_sizeof_args() == sizeof f, 10);
  qknr_rms_args_init(&n);
  CHECK(qknr_rms_forward(&n, NULL) == QKNR_ERR_UNSUPPORTED, 20);     /* hidden 0 */
  n.hidden = 128; n.flags = QKNR_RMS_UNIT_OFFSET; n.out = QKNR_RMS_OUT_E4M3; n.scale_block = 128;
  CHECK(qknr_rms_forward(&n, NULL) == QKNR_OK && qknr_rms_backward(&n, NULL) == QKNR_OK, 21);
  n.tokens = 1000;
  CHECK(qknr_rms_workspace_bytes(&n, &bytes) == QKNR_OK && bytes > 0, 22);
  CHECK(qknr_rms_backward(&n, NULL) == QKNR_ERR_NULL, 23);
  qknr_pack_args_init(&p);
  CHECK(qknr_pack_forward(&p, NULL) == QKNR_ERR_UNSUPPORTED, 30);    /* head_dim 0 */
  p.head_dim = 64; p.n_heads_q = 4; p.n_heads_k = 2;
  CHECK(qknr_pack_forward(&p, NULL) == QKNR_OK && qknr_pack_backward(&p, NULL) == QKNR_OK, 31);
  p.batch = 3; p.rows_q = p.rows_k = 5000;
  CHECK(qknr_pack_workspace_bytes(&p, &bytes) == QKNR_OK && bytes > 0, 32);
  CHECK(qknr_pack_backward_workspace_bytes(&p, &bytes) == QKNR_OK && bytes >= 4 * 5000 * sizeof(float), 33);
  CHECK(qknr_pack_forward(&p, NULL) == QKNR_ERR_NULL, 34);
  qknr_prefix_args_init(&f);
  CHECK(qknr_prefix_forward(&f, NULL) == QKNR_ERR_UNSUPPORTED, 40);
  f.head_dim = 128; f.n_heads_q = 4; f.n_heads_k = 2; f.batch = 64; f.prefix = 9000;
  CHECK(qknr_prefix_forward(&f, NULL) == QKNR_ERR_NULL, 41);         /* no prefix_k */
  f.seq_q = 1;
  CHECK(qknr_prefix_workspace_bytes(&f, &bytes) == QKNR_OK && bytes > 0, 42);
  puts("ok");
  return 0;
}
"""


def test_c99_program_links_and_runs(tmp_path, built_lib):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe, libdir = tmp_path / "abi.c", tmp_path / "abi", os.path.dirname(built_lib)
    src.write_text(PROGRAM)
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I" + INCLUDE, str(src), "-o", str(exe),
                        "-L" + libdir, "-lqknr", "-Wl,-rpath," + libdir, "-Wl,-rpath," + B.cuda_lib_dir()],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", (run.returncode, run.stdout, run.stderr)


def test_short_packed_calls_need_no_workspace(lib):  # noqa: F811
    n = ctypes.c_size_t(7)
    a = changed(pack, dict(rows_q=240, rows_k=240))
    assert lib.qknr_pack_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value == 0
