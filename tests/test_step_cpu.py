"""include/qstep.h without a GPU: exports, the refusal of bad arguments by
status before any CUDA call, and the Python binding's own checks."""
import ctypes
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

import ggml_block_quantized_gb300 as qg  # noqa: E402
from ggml_block_quantized_gb300 import step  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_TYPE, ERR_SHAPE, ERR_ALIGN, ERR_NULL = 0, -1, -2, -3, -4
A, B, C = 0x10000, 0x20000, 0x30000


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return step._lib()


def test_declarations_are_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qstep.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M)))
    assert names == sorted(qg.STEP_SYMBOLS)
    out = subprocess.run(["nm", "-D", "--defined-only", qg.library_path()], capture_output=True, text=True).stdout
    assert set(names) <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def norm_args(**kw):
    a = dict(h=A, y=B, h_stride=256, y_stride=256, post_w=None, post_b=None, gate=None, gate_stride=0, w=C, b=None, h_out=A,
             h_out_stride=256, x_out=C, xq=None, n=3, d=256, h_type=0, y_type=0, x_type=0, act_type=8, layer=0, scale=1.0,
             eps=1e-5)
    a.update(kw)
    return step._NormArgs(*[a[n] for n, _ in step._NormArgs._fields_])


@pytest.mark.parametrize("want,kw", [
    (ERR_TYPE, dict(h_type=2)), (ERR_TYPE, dict(y_type=-1)), (ERR_TYPE, dict(x_type=8)), (ERR_TYPE, dict(xq=A, act_type=2)),
    (ERR_SHAPE, dict(n=-1)), (ERR_SHAPE, dict(n=(1 << 30) + 1)), (ERR_SHAPE, dict(d=0)), (ERR_SHAPE, dict(d=16385)),
    (ERR_SHAPE, dict(h_stride=-1)), (ERR_SHAPE, dict(y_stride=-256)), (ERR_SHAPE, dict(gate_stride=-4)),
    (ERR_SHAPE, dict(h_out_stride=255)), (ERR_SHAPE, dict(scale=float("nan"))), (ERR_SHAPE, dict(scale=float("inf"))),
    (ERR_SHAPE, dict(eps=-1.0)), (ERR_SHAPE, dict(eps=float("nan"))), (ERR_SHAPE, dict(xq=A, act_type=15, d=224)),
    (ERR_SHAPE, dict(xq=A, act_type=9, d=250)), (ERR_NULL, dict(h=None)), (ERR_NULL, dict(h_out=None, x_out=None)),
    (ERR_ALIGN, dict(h=A + 2)), (ERR_ALIGN, dict(y=B + 1, y_type=1)), (ERR_ALIGN, dict(w=C + 2)), (ERR_ALIGN, dict(b=C + 1)),
    (ERR_ALIGN, dict(gate=A + 3)), (ERR_ALIGN, dict(post_w=A + 2)), (ERR_ALIGN, dict(h_out=A + 1)), (ERR_ALIGN, dict(x_out=C + 2)),
    (ERR_ALIGN, dict(xq=A + 8)), (ERR_ALIGN, dict(xq=A, h=A + 4)), (ERR_ALIGN, dict(xq=A, y_stride=258)),
    (ERR_ALIGN, dict(xq=A, h_type=1, h_stride=260)), (ERR_ALIGN, dict(xq=A, w=C + 8)), (OK, dict(n=0, h=None)),
])
def test_norm_refusals(L, want, kw):
    assert L.qnorm_residual(ctypes.byref(norm_args(**kw)), None) == want


def test_norm_without_arguments(L):
    assert L.qnorm_residual(None, None) == ERR_NULL


@pytest.mark.parametrize("want,kw", [
    (ERR_TYPE, dict(type=2)), (ERR_SHAPE, dict(n=-1)), (ERR_SHAPE, dict(n=(1 << 24) + 1)), (ERR_SHAPE, dict(vocab=0)),
    (ERR_SHAPE, dict(vocab=(1 << 19) + 1)), (ERR_SHAPE, dict(stride=-1)), (ERR_NULL, dict(logits=None)),
    (ERR_NULL, dict(uniform=None)), (ERR_NULL, dict(token=None)), (ERR_ALIGN, dict(logits=A + 2)),
    (ERR_ALIGN, dict(type=1, logits=A + 1)), (ERR_ALIGN, dict(uniform=A + 2)), (ERR_ALIGN, dict(token=A + 1)),
    (ERR_ALIGN, dict(prob=A + 2)), (ERR_ALIGN, dict(temperature=A + 2)), (ERR_ALIGN, dict(top_k=A + 2)),
    (ERR_ALIGN, dict(top_p=A + 2)), (ERR_ALIGN, dict(min_p=A + 2)), (OK, dict(n=0, logits=None)),
])
def test_sample_refusals(L, want, kw):
    a = dict(type=0, logits=A, stride=100, n=2, vocab=100, temperature=None, top_k=None, top_p=None, min_p=None, uniform=B,
             token=C, prob=None)
    a.update(kw)
    assert L.qsample(*a.values(), None) == want


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 64)
    with pytest.raises(TypeError):
        qg.norm_residual(x, x)
    with pytest.raises(TypeError):
        qg.sample_tokens(x, torch.zeros(2))
    with pytest.raises(TypeError):
        qg.norm_residual(None)
    with pytest.raises(TypeError):
        qg.sample_tokens([[1.0]], None)


class Tensor(torch.Tensor):
    """Says that it lies on the GPU: the binding's checks alone are meant."""
    is_cuda = True

    def get_device(self):
        return 0


@pytest.fixture
def fake(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(step, "_stream", lambda stream, device: None)
    return lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype).as_subclass(Tensor)


def test_norm_binding_checks(L, fake):
    h, y, w = fake(2, 64), fake(2, 64), fake(64)
    new = dict(h_out=fake(2, 64), x_out=fake(2, 64))
    for bad, kw in ((ValueError, dict(y=fake(2, 63))), (TypeError, dict(y=fake(2, 64, dtype=torch.float64))),
                    (ValueError, dict(weight=fake(63))), (TypeError, dict(weight=fake(64, dtype=torch.float16))),
                    (ValueError, dict(gate=fake(2, 63))), (ValueError, dict(gate=fake(63))), (ValueError, dict(y=None, gate=w)),
                    (ValueError, dict(y=None, post_weight=w)), (ValueError, dict(post_bias=w)), (ValueError, dict(weight=None, bias=w)),
                    (TypeError, dict(h_out=fake(2, 64, dtype=torch.float16))), (ValueError, dict(h_out=fake(3, 64))),
                    (ValueError, dict(x_out=fake(2, 128)[:, :64])), (ValueError, dict(x_out=fake(64, 2).t())),
                    (ValueError, dict(y=fake(64, 2).t())), (ValueError, dict(xq=fake(999, dtype=torch.uint8))),
                    (ValueError, dict(xq=fake(67, dtype=torch.uint8), act_type=qg.Q8_0)),
                    (ValueError, dict(xq=fake(999, dtype=torch.uint8), act_type=qg.Q8_K)),
                    (ValueError, dict(xq=fake(999, dtype=torch.uint8), act_type=qg.Q4_0)),
                    (TypeError, dict(xq=fake(999), act_type=qg.Q8_0)), (ValueError, dict(act_type=qg.Q8_0))):
        with pytest.raises(bad):
            qg.norm_residual(h, **{**dict(y=y, weight=w), **new, **kw})
    with pytest.raises(ValueError):
        qg.norm_residual(fake(64))


def test_sample_binding_checks(L, fake):
    x, u = fake(3, 50), fake(3)
    out = dict(out=fake(3, dtype=torch.int32))
    for bad, kw in ((ValueError, dict(uniform=fake(2))), (TypeError, dict(uniform=fake(3, dtype=torch.float64))),
                    (TypeError, dict(uniform=None)), (ValueError, dict(temperature=fake(1))), (TypeError, dict(temperature=1.0)),
                    (TypeError, dict(top_k=fake(3))), (ValueError, dict(top_k=fake(4, dtype=torch.int32))),
                    (ValueError, dict(top_p=fake(3, 1))), (TypeError, dict(min_p=fake(3, dtype=torch.float16))),
                    (TypeError, dict(out=fake(3))), (ValueError, dict(prob_out=fake(6)[::2])), (ValueError, dict(logits=fake(50))),
                    (ValueError, dict(logits=fake(50, 3).t())), (TypeError, dict(logits=fake(3, 50, dtype=torch.bfloat16)))):
        with pytest.raises(bad):
            qg.sample_tokens(**{**dict(logits=x, uniform=u), **out, **kw})
