"""What the training operators' C entry points and their binding refuse, each
before any CUDA call.  Runs without a GPU: the addresses here are plain
integers that are never touched, because every call returns during
validation (or has nothing to launch)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from diffusion_transformer_qk_gb300 import build as B
from diffusion_transformer_qk_gb300 import qknr as Q

# never where a GPU is visible: a call that validation let through by mistake
# must not reach a device with these addresses
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only tests with fake device addresses")

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
FAKE, STEP = 1 << 40, 1 << 30         # 16-byte aligned; tensors a GB apart do not meet
NULL, SHAPE, ALIGN, UNSUPPORTED, OVERLAP, ABI = 1, 2, 3, 4, 7, 8


@pytest.fixture(scope="module")
def lib(built_lib):
    return Q.load()


def fake(n):
    return FAKE + n * STEP


def refused(lib, fn, a, expect):
    st = getattr(lib, fn)(ctypes.byref(a), None)
    msg = lib.qknr_last_error().decode()
    assert st == expect, (st, msg)
    assert msg


def changed(make, change):
    a = make()
    for name, value in change.items():
        setattr(a, name, value)
    return a


def test_struct_layouts_match(lib):
    assert lib.qknr_ln_sizeof_args() == ctypes.sizeof(Q.QknrLnArgs)
    assert lib.qknr_sizeof_grad_args() == ctypes.sizeof(Q.QknrGradArgs)
    assert lib.qknr_attn_sizeof_args() == ctypes.sizeof(Q.QknrAttnArgs)


@pytest.mark.parametrize("struct,init,defaults", [
    ("QknrLnArgs", "qknr_ln_args_init", dict(dtype=Q.BF16, param_dtype=Q.FP32)),
    ("QknrGradArgs", "qknr_grad_args_init", dict(dtype=Q.BF16, cos_dtype=Q.FP32, cos_layout=0, rope_style=0)),
    ("QknrAttnArgs", "qknr_attn_args_init", dict(dtype=Q.BF16, causal=0, scale=0.0)),
])
def test_init_writes_every_field(lib, struct, init, defaults):
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


@pytest.mark.parametrize("fn", ["qknr_ln_forward", "qknr_ln_backward", "qknr_backward", "qknr_attn_forward", "qknr_attn_backward"])
def test_null_args(lib, fn):
    assert getattr(lib, fn)(None, None) == NULL


@pytest.mark.parametrize("fn,make", [
    ("qknr_ln_workspace_bytes", lambda: ln()), ("qknr_grad_workspace_bytes", lambda: grad()),
    ("qknr_attn_workspace_bytes", lambda: attn()), ("qknr_attn_backward_workspace_bytes", lambda: attn()),
])
def test_workspace_queries(lib, fn, make):
    n = ctypes.c_size_t(7)
    assert getattr(lib, fn)(None, ctypes.byref(n)) == NULL and n.value == 0
    assert getattr(lib, fn)(ctypes.byref(make()), None) == NULL
    assert getattr(lib, fn)(ctypes.byref(make()), ctypes.byref(n)) == 0 and n.value > 0
    a = changed(make, dict(dtype=9))
    assert getattr(lib, fn)(ctypes.byref(a), ctypes.byref(n)) == UNSUPPORTED and n.value == 0


# ---------------------------------------------------------------------------
# layer norm

def ln(T=600, C=1536):
    a = Q.QknrLnArgs()
    Q.load().qknr_ln_args_init(ctypes.byref(a))
    a.x, a.y, a.weight, a.bias, a.mean, a.rstd, a.dy, a.dx = (fake(i) for i in range(8))
    a.dweight, a.dbias, a.workspace, a.workspace_bytes = fake(8), fake(9), fake(10), STEP
    a.tokens, a.hidden = T, C
    return a


LN_BOTH = [
    (dict(abi_version=99), ABI), (dict(dtype=Q.FP32), UNSUPPORTED), (dict(param_dtype=Q.FP16), UNSUPPORTED),
    (dict(hidden=0), UNSUPPORTED), (dict(hidden=1540), UNSUPPORTED), (dict(hidden=32776), UNSUPPORTED),
    (dict(tokens=-1), SHAPE), (dict(rows_per_batch=-1), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(x=None), NULL), (dict(x_stride=1528), SHAPE), (dict(param_stride=8), SHAPE), (dict(x_stride=1540), ALIGN),
    (dict(x=FAKE + 8), ALIGN), (dict(weight=FAKE + 4), ALIGN), (dict(bias=FAKE + 4), ALIGN),
    (dict(param_stride=1538), ALIGN), (dict(mean=FAKE + 2), ALIGN), (dict(rstd=FAKE + 1), ALIGN),
]


@pytest.mark.parametrize("change,expect", LN_BOTH + [
    (dict(y_stride=8), SHAPE), (dict(y=FAKE + STEP + 2), ALIGN), (dict(y_stride=1540), ALIGN),
    (dict(y=FAKE + 16), OVERLAP), (dict(y=FAKE, y_stride=1544), OVERLAP), (dict(y=fake(2)), OVERLAP),
    (dict(y=fake(3)), OVERLAP), (dict(y=fake(4)), OVERLAP), (dict(y=fake(5)), OVERLAP),
])
def test_layer_norm_refuses(lib, change, expect):
    refused(lib, "qknr_ln_forward", changed(ln, change), expect)


@pytest.mark.parametrize("change,expect", LN_BOTH + [
    (dict(dy=None), NULL), (dict(mean=None), NULL), (dict(rstd=None), NULL), (dict(dy_stride=8), SHAPE),
    (dict(dx_stride=8), SHAPE), (dict(dy=FAKE + 6 * STEP + 8), ALIGN), (dict(dx=FAKE + 7 * STEP + 8), ALIGN),
    (dict(dweight=FAKE + 8 * STEP + 4), ALIGN), (dict(dbias=FAKE + 9 * STEP + 8), ALIGN),
    (dict(workspace=None), NULL), (dict(workspace_bytes=16), SHAPE), (dict(workspace=FAKE + 10 * STEP + 8), ALIGN),
    (dict(dx=FAKE + 6 * STEP + 16), OVERLAP), (dict(dx=FAKE), OVERLAP), (dict(dweight=fake(6)), OVERLAP),
    (dict(dbias=fake(8)), OVERLAP), (dict(workspace=fake(7)), OVERLAP), (dict(workspace=FAKE), OVERLAP),
    (dict(dweight=fake(2)), OVERLAP),
])
def test_layer_norm_backward_refuses(lib, change, expect):
    refused(lib, "qknr_ln_backward", changed(ln, change), expect)


def test_layer_norm_without_rows_needs_nothing(lib):
    a = Q.QknrLnArgs()
    lib.qknr_ln_args_init(ctypes.byref(a))
    a.hidden = 64
    assert lib.qknr_ln_forward(ctypes.byref(a), None) == 0
    assert lib.qknr_ln_backward(ctypes.byref(a), None) == 0


# ---------------------------------------------------------------------------
# the backward pass of QK-RMSNorm + RoPE

def grad(T=64, H=4, D=128):
    a = Q.QknrGradArgs()
    Q.load().qknr_grad_args_init(ctypes.byref(a))
    row = 3 * H * D
    for name, base in (("q", 0), ("dq", 1), ("dq_out", 2)):
        setattr(a, name, fake(base))
        setattr(a, name.replace("q", "k", 1), fake(base) + H * D * 2)
        setattr(a, name + "_stride", row)
        setattr(a, name.replace("q", "k", 1) + "_stride", row)
    a.dv, a.dv_out = fake(1) + 2 * H * D * 2, fake(2) + 2 * H * D * 2
    a.dv_stride = a.dv_out_stride = row
    a.tokens, a.n_heads_q, a.n_heads_k, a.n_heads_v, a.head_dim = T, H, H, H, D
    a.gamma_q, a.gamma_k, a.cos, a.sin, a.dgamma_q, a.dgamma_k = (fake(i) for i in range(3, 9))
    a.workspace, a.workspace_bytes = fake(9), STEP
    return a


ROW = 4 * 128 * 2                     # bytes of one tensor's columns in a packed row


@pytest.mark.parametrize("change,expect", [
    (dict(abi_version=99), ABI), (dict(dtype=Q.FP32), UNSUPPORTED), (dict(cos_dtype=Q.FP16), UNSUPPORTED),
    (dict(cos_layout=2), UNSUPPORTED), (dict(rope_style=2), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(tokens=-1), SHAPE), (dict(cos_rows=-1), SHAPE), (dict(n_heads_q=-1), SHAPE), (dict(n_heads_v=-1), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(cos_layout=1, n_heads_k=2), SHAPE), (dict(gamma_q=None), NULL), (dict(q=None), NULL),
    (dict(dk=None), NULL), (dict(cos=None), NULL), (dict(sin=None), NULL), (dict(dv=None), NULL),
    (dict(workspace=None), NULL), (dict(workspace_bytes=64), SHAPE), (dict(workspace=FAKE + 9 * STEP + 4), ALIGN),
    (dict(q_stride=8), SHAPE), (dict(dk_stride=8), SHAPE), (dict(dq_out_stride=8), SHAPE), (dict(dv_stride=8), SHAPE),
    (dict(q=FAKE + 8), ALIGN), (dict(dq=fake(1) + 2), ALIGN), (dict(dk_out_stride=3 * 512 + 4), ALIGN),
    (dict(cos=fake(5) + 4), ALIGN), (dict(gamma_q=fake(3) + 2), ALIGN), (dict(dgamma_k=fake(8) + 2), ALIGN),
    (dict(dv=fake(1) + 2 * ROW + 8), ALIGN),
    (dict(dq_out=FAKE), OVERLAP),                       # onto q
    (dict(dq_out=fake(1) + ROW), OVERLAP),              # onto dk
    (dict(dk_out=fake(2)), OVERLAP),                    # onto dq_out
    (dict(dq_out=None, dk_out=fake(1)), OVERLAP),       # dq stays in place, dk_out is put there
    (dict(dq_out=None, dk_out=None, dk=fake(1)), OVERLAP),   # two gradients in one place, both in place
    (dict(dgamma_q=fake(5)), OVERLAP), (dict(dgamma_q=fake(8)), OVERLAP), (dict(workspace=fake(2)), OVERLAP),
    (dict(dgamma_k=fake(1)), OVERLAP), (dict(dv_out=FAKE), OVERLAP),
])
def test_qk_backward_refuses(lib, change, expect):
    refused(lib, "qknr_backward", changed(grad, change), expect)


def test_qk_backward_without_work_is_ok(lib):
    a = Q.QknrGradArgs()
    lib.qknr_grad_args_init(ctypes.byref(a))
    a.head_dim = 64
    assert lib.qknr_backward(ctypes.byref(a), None) == 0
    b = grad()
    b.n_heads_q = b.n_heads_k = 0
    b.dv_out = None
    assert lib.qknr_backward(ctypes.byref(b), None) == 0


# ---------------------------------------------------------------------------
# attention

def attn(B=2, Sq=100, Sk=1000, Hq=4, Hk=4, D=128):
    """Packed columns in and out; keys enough that both passes want a workspace."""
    a = Q.QknrAttnArgs()
    Q.load().qknr_attn_args_init(ctypes.byref(a))
    row = (Hq + 2 * Hk) * D
    for base, names in ((0, "q k v"), (1, "dq dk dv")):
        for i, name in enumerate(names.split()):
            setattr(a, name, fake(base) + i * Hq * D * 2)
            setattr(a, name + "_stride", row)
    a.o, a.lse, a.dout, a.q_lens, a.k_lens, a.workspace, a.workspace_bytes = (*(fake(i) for i in range(2, 8)), STEP)
    a.batch, a.seq_q, a.seq_k, a.n_heads_q, a.n_heads_k, a.head_dim = B, Sq, Sk, Hq, Hk, D
    return a


ATTN_BOTH = [
    (dict(abi_version=99), ABI), (dict(dtype=Q.FP32), UNSUPPORTED), (dict(head_dim=32), UNSUPPORTED),
    (dict(head_dim=256), UNSUPPORTED), (dict(batch=-1), SHAPE), (dict(seq_q=-1), SHAPE), (dict(seq_k=-1), SHAPE),
    (dict(n_heads_q=0), SHAPE), (dict(n_heads_k=0), SHAPE), (dict(n_heads_q=6), SHAPE), (dict(scale=-1.0), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(seq_q=1 << 30, batch=8), UNSUPPORTED),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(o=None), NULL), (dict(lse=None), NULL),
    (dict(q_stride=8), SHAPE), (dict(v_stride=8), SHAPE), (dict(o_stride=8), SHAPE), (dict(k_stride=1 << 31), UNSUPPORTED),
    (dict(k_stride=1540), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(o=fake(2) + 4), ALIGN), (dict(lse=fake(3) + 2), ALIGN),
    (dict(q_lens=fake(5) + 1), ALIGN), (dict(k_lens=fake(6) + 2), ALIGN), (dict(workspace=None), NULL),
    (dict(workspace_bytes=64), SHAPE), (dict(workspace=fake(7) + 4), ALIGN), (dict(workspace=FAKE), OVERLAP),
    (dict(workspace=fake(5)), OVERLAP),
]


@pytest.mark.parametrize("change,expect", ATTN_BOTH + [
    (dict(o=FAKE), OVERLAP), (dict(o=fake(5)), OVERLAP), (dict(lse=FAKE), OVERLAP), (dict(lse=fake(2)), OVERLAP),
    (dict(workspace=fake(2)), OVERLAP), (dict(workspace=fake(3)), OVERLAP),
])
def test_attention_refuses(lib, change, expect):
    refused(lib, "qknr_attn_forward", changed(attn, change), expect)


@pytest.mark.parametrize("change,expect", ATTN_BOTH + [
    (dict(dout=None), NULL), (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dv=None), NULL),
    (dict(dout=fake(4) + 8), ALIGN), (dict(dk_stride=8), SHAPE), (dict(dv_stride=1540), ALIGN),
    (dict(dq=FAKE), OVERLAP), (dict(dk=fake(2)), OVERLAP), (dict(dv=fake(3)), OVERLAP), (dict(dq=fake(4)), OVERLAP),
    (dict(workspace=fake(1)), OVERLAP), (dict(workspace=fake(3)), OVERLAP),
    (dict(dv=fake(1) + ROW), OVERLAP),                  # onto dk
    (dict(dk=fake(1) + ROW - 16), OVERLAP),             # its first columns onto dq's last
    (dict(dq=fake(1) + 16), OVERLAP),
    (dict(dq_stride=2048), OVERLAP),                    # another stride in the same place
])
def test_attention_backward_refuses(lib, change, expect):
    refused(lib, "qknr_attn_backward", changed(attn, change), expect)


def test_attention_without_work_needs_nothing(lib):
    a = Q.QknrAttnArgs()
    lib.qknr_attn_args_init(ctypes.byref(a))
    a.head_dim, a.n_heads_q, a.n_heads_k = 64, 4, 2
    for b, sq, sk in ((0, 5, 5), (3, 0, 0)):
        a.batch, a.seq_q, a.seq_k = b, sq, sk
        assert lib.qknr_attn_forward(ctypes.byref(a), None) == 0
        assert lib.qknr_attn_backward(ctypes.byref(a), None) == 0


# ---------------------------------------------------------------------------
# the binding: tensors on the CPU, wrong shapes and types

def act(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: Q.layer_norm(act(4, 64)),                                            # not on a GPU
    lambda: Q.layer_norm(act(4, 64, dtype=torch.float32)),
    lambda: Q.layer_norm(act(2, 4, 64)),
    lambda: Q.layer_norm_backward(act(4, 64), act(4, 64), None, act(4), act(4)),
    lambda: Q.attention(act(4, 128), act(4, 128), act(4, 128, dtype=torch.float16), 1, 1, 128),
    lambda: Q.attention(act(4, 128), act(4, 128), act(4, 128), 1, 1, 128),       # not on a GPU
    lambda: Q.attention(act(0, 128), act(0, 64), act(0, 128), 1, 1, 128),        # width
    lambda: Q.attention(act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, batch=0),
    lambda: Q.attention(act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, scale=0.0),
    lambda: Q.attention(act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, scale=-2.0),
    lambda: Q.attention(act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, scale=float("inf")),
    lambda: Q.attention(act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, scale=1e-60),   # zero in fp32
    lambda: Q.attention(act(0, 128), act(0, 128), act(0, 128), 1, 1, 128, k_lens=torch.zeros(1, dtype=torch.int32)),
    lambda: Q.attention_backward(act(0, 64), act(0, 128), act(0, 128), act(0, 128), act(0, 128), None, 1, 1, 128),
    lambda: Q.qk_norm_rope_packed_backward(act(4, 384), act(4, 384), 1, 1, 1, 128, None, None, act(4, 64), act(4, 64)),
    lambda: Q.qk_norm_rope_packed_backward(act(4, 300), act(4, 300), 1, 1, 1, 128, None, None, act(4, 128), act(4, 128)),
    lambda: Q.qk_norm_rope_packed_backward(act(4, 256), act(4, 384), 1, 1, 1, 128, None, None, act(4, 128), act(4, 128)),
    lambda: Q.qk_norm_rope_packed_backward(act(4, 384), act(4, 384), 1, 1, 1, 128, None, None, act(4, 128), act(4, 128)),
])
def test_binding_refuses(lib, call):
    with pytest.raises(ValueError):
        call()


def test_binding_checks_what_it_puts_in():
    with pytest.raises(ValueError):
        Q._workspace(attn(), None, torch.zeros(64), None, None)
    with pytest.raises(ValueError):
        Q._status(attn(), True, torch.zeros(1, dtype=torch.int32), None)
    with pytest.raises(ValueError):
        Q._vector(torch.zeros(4), 4, "lse")


# ---------------------------------------------------------------------------
# C

PROGRAM = r"""
#include <stdio.h>
#include "qknr_ln.h"
#include "qknr_grad.h"
#include "qknr_attn.h"

#define CHECK(cond, code) do { if (!(cond)) { fprintf(stderr, "failed: %s\n", #cond); return code; } } while (0)

int main(void) {
  qknr_ln_args n;
  qknr_grad_args g;
  qknr_attn_args a;
  size_t bytes = 0;
  CHECK(qknr_ln_sizeof_args() == sizeof n && qknr_sizeof_grad_args() == sizeof g && qknr_attn_sizeof_args() == sizeof a, 10);
  qknr_ln_args_init(&n);
  CHECK(qknr_ln_forward(&n, NULL) == QKNR_ERR_UNSUPPORTED, 20);      /* hidden 0 */
  n.hidden = 64; n.flags = QKNR_LN_UNIT_OFFSET;
  CHECK(qknr_ln_forward(&n, NULL) == QKNR_OK && qknr_ln_backward(&n, NULL) == QKNR_OK, 21);
  n.tokens = 1000;
  CHECK(qknr_ln_workspace_bytes(&n, &bytes) == QKNR_OK && bytes > 0, 22);
  CHECK(qknr_ln_backward(&n, NULL) == QKNR_ERR_NULL, 23);
  qknr_grad_args_init(&g);
  CHECK(qknr_backward(&g, NULL) == QKNR_ERR_UNSUPPORTED, 30);        /* head_dim 0 */
  g.head_dim = 128; g.n_heads_q = 4; g.tokens = 9;
  CHECK(qknr_grad_workspace_bytes(&g, &bytes) == QKNR_OK && bytes >= 2 * 128 * sizeof(float), 31);
  CHECK(qknr_backward(&g, NULL) == QKNR_ERR_NULL, 32);
  qknr_attn_args_init(&a);
  CHECK(qknr_attn_forward(&a, NULL) == QKNR_ERR_UNSUPPORTED, 40);
  a.head_dim = 64; a.n_heads_q = 4; a.n_heads_k = 2;
  CHECK(qknr_attn_forward(&a, NULL) == QKNR_OK && qknr_attn_backward(&a, NULL) == QKNR_OK, 41);
  a.batch = 1; a.seq_q = a.seq_k = 300;
  CHECK(qknr_attn_workspace_bytes(&a, &bytes) == QKNR_OK, 42);
  CHECK(qknr_attn_backward_workspace_bytes(&a, &bytes) == QKNR_OK && bytes >= 4 * 300 * sizeof(float), 43);
  CHECK(qknr_attn_forward(&a, NULL) == QKNR_ERR_NULL, 44);
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
