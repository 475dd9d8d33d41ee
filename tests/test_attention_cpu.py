"""include/qattn.h without a GPU: exports, sizes, the refusal of bad arguments
by status before any CUDA call, and the Python binding's own checks."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref  # noqa: E402
import ggml_block_quantized_gb300 as qg  # noqa: E402
from ggml_block_quantized_gb300 import attention as at  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_TYPE, ERR_SHAPE, ERR_ALIGN, ERR_NULL, ERR_WS = 0, -1, -2, -3, -4, -7
A, B, C, MIS = 0x10000, 0x20000, 0x30000, 0x10008


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return at._lib()


def test_declarations_are_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qattn.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M)))
    assert names == sorted(qg.ATTENTION_SYMBOLS)
    out = subprocess.run(["nm", "-D", "--defined-only", qg.library_path()], capture_output=True, text=True).stdout
    assert set(names) <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def test_cache_bytes(L):
    assert qg.kv_cache_bytes(3, 8, 128, 64) == 3 * 64 * 8 * (2 * 128 // 32 * 18)  # Q4_0's 18 bytes a block
    assert qg.kv_cache_bytes(5, 1, 64, 16) == 5 * 16 * 72
    assert qg.kv_cache_bytes(0, 1, 64, 16) == 0
    assert qg.kv_cache_bytes(1 << 24, 64, 128, 64) == (1 << 30) * 64 * 144  # past 32 bits
    for bad in ((-1, 8, 128, 64), (1, 0, 128, 64), (1, 8, 96, 64), (1, 8, 128, 24), (1, 8, 128, 0), (1 << 31, 8, 128, 64)):
        assert qg.kv_cache_bytes(*bad) == -1


def test_layout_is_a_permutation():
    """Every byte of a group belongs to one row's codes or scales."""
    for d in (64, 128):
        seen = np.concatenate([x.ravel() for i in range(16) for x in attn_ref.slot_bytes(16, 1, d, i, 0)])
        assert np.array_equal(np.sort(seen), np.arange(18 * d))


def cache(data=A, n_pages=4, heads=2, d=128, page=16):
    return at._Cache(data, n_pages, heads, d, page)


def append_args(**kw):
    a = dict(q=None, k=A, v=B, q_stride=1024, k_stride=256, v_stride=256, slots=C, positions=C, rope=None, q_out=None,
             k_out=None, v_out=None, n_tok=3, n_heads=8, in_type=0, out_type=0, n_pos=16, rot_dim=128, rope_pairs=0)
    a.update(kw)
    return at._AppendArgs(*[a[n] for n, _ in at._AppendArgs._fields_])


@pytest.mark.parametrize("want,kw", [
    (ERR_TYPE, dict(in_type=8)), (ERR_TYPE, dict(out_type=2)), (ERR_SHAPE, dict(n_tok=-1)),
    (ERR_SHAPE, dict(q=A, q_out=B, n_heads=7)), (ERR_SHAPE, dict(rope=A, rot_dim=12)),
    (ERR_SHAPE, dict(rope=A, rot_dim=136)), (ERR_SHAPE, dict(rope=A, n_pos=-1)), (ERR_SHAPE, dict(n_tok=1 << 30)),
    (ERR_NULL, dict(k=None)), (ERR_NULL, dict(v=None)), (ERR_NULL, dict(slots=None)), (ERR_NULL, dict(q=A)),
    (ERR_NULL, dict(rope=A, positions=None)), (ERR_ALIGN, dict(k=MIS)), (ERR_ALIGN, dict(q=MIS, q_out=A)),
    (ERR_ALIGN, dict(rope=MIS)), (ERR_ALIGN, dict(k_out=MIS)), (ERR_ALIGN, dict(slots=C + 2)),
    (ERR_SHAPE, dict(k_stride=252)), (ERR_SHAPE, dict(v_stride=258)), (ERR_SHAPE, dict(in_type=1, k_stride=260)),
    (ERR_SHAPE, dict(k_stride=0)), (OK, dict(n_tok=0, k=None)),
])
def test_append_refusals(L, want, kw):
    assert L.qkv_append(ctypes.byref(cache()), ctypes.byref(append_args(**kw)), None) == want


def test_cache_refusals(L):
    good = append_args()
    assert L.qkv_append(None, ctypes.byref(good), None) == ERR_NULL
    assert L.qkv_append(ctypes.byref(cache()), None, None) == ERR_NULL
    assert L.qkv_append(ctypes.byref(cache(d=80)), ctypes.byref(good), None) == ERR_SHAPE
    assert L.qkv_append(ctypes.byref(cache(page=20)), ctypes.byref(good), None) == ERR_SHAPE
    assert L.qkv_append(ctypes.byref(cache(data=None)), ctypes.byref(good), None) == ERR_NULL
    assert L.qkv_append(ctypes.byref(cache(data=MIS)), ctypes.byref(good), None) == ERR_ALIGN
    c = ctypes.byref(cache())
    assert L.qkv_read(c, A, -1, B, C, None) == ERR_SHAPE
    assert L.qkv_read(c, None, 2, B, C, None) == ERR_NULL
    assert L.qkv_read(c, A, 2, MIS, C, None) == ERR_ALIGN
    assert L.qkv_read(c, A, 0, B, C, None) == OK
    assert L.qkv_read(c, A, 2, None, None, None) == OK


ATTEND = dict(type=0, q=A, q_stride=1024, out=B, table=C, table_stride=4, lengths=C, q_offsets=None, n_seq=2, n_tok=2,
              n_heads=8, max_q_len=1, scale=0.1, workspace=A, workspace_bytes=1 << 40)


@pytest.mark.parametrize("want,kw", [
    (ERR_TYPE, dict(type=2)), (ERR_SHAPE, dict(n_heads=7)), (ERR_SHAPE, dict(n_heads=0)), (ERR_SHAPE, dict(n_seq=-1)),
    (ERR_SHAPE, dict(max_q_len=0)), (ERR_SHAPE, dict(max_q_len=1 << 30)), (ERR_SHAPE, dict(table_stride=-1)),
    (ERR_SHAPE, dict(n_tok=1)), (ERR_SHAPE, dict(scale=float("nan"))), (ERR_SHAPE, dict(scale=float("inf"))),
    (ERR_SHAPE, dict(q_stride=1020)), (ERR_SHAPE, dict(q_stride=1026)), (ERR_NULL, dict(q=None)),
    (ERR_NULL, dict(out=None)), (ERR_NULL, dict(lengths=None)), (ERR_NULL, dict(table=None)), (ERR_ALIGN, dict(q=MIS)),
    (ERR_ALIGN, dict(out=MIS)), (ERR_ALIGN, dict(workspace=MIS)), (ERR_ALIGN, dict(lengths=C + 1)),
    (ERR_WS, dict(workspace=None)), (ERR_WS, dict(workspace_bytes=15)), (OK, dict(n_seq=0, n_tok=0)),
])
def test_attend_refusals(L, want, kw):
    a = {**ATTEND, **kw}
    assert L.qkv_attend(ctypes.byref(cache()), *a.values(), None) == want


def test_sizes_whose_products_pass_64_bits(L):
    """They are refused like other sizes out of range, before any of them is multiplied."""
    for stride in (1 << 31, 1 << 59, (1 << 63) - 1):
        assert L.qkv_attend(ctypes.byref(cache()), *{**ATTEND, "table_stride": stride}.values(), None) == ERR_SHAPE
    for n in ((1 << 62) + 1, (1 << 63) - 1):
        assert L.qkv_append(ctypes.byref(cache()), ctypes.byref(append_args(n_tok=n)), None) == ERR_SHAPE
        assert L.qkv_read(ctypes.byref(cache()), A, n, B, C, None) == ERR_SHAPE


def test_attend_workspace(L):
    ws = L.qkv_attend_workspace_bytes
    assert ws(128, 8, 32, 1) >= 16 and ws(64, 8, 8, 4) >= 16
    assert ws(128, 8, 32, 8) >= ws(128, 8, 32, 1)
    for bad in ((96, 8, 32, 1), (128, 0, 32, 1), (128, 8, 31, 1), (128, 8, 32, 0), (128, 1, 1024, 1 << 20)):
        assert ws(*bad) == 0


PROMPT = dict(q=A, q_stride=1024, k=B, k_stride=256, v=C, v_stride=256, out_type=1, out=A, offsets=C, n_seq=1, n_tok=5,
              n_heads=8, n_kv_heads=2, head_dim=128, scale=0.1)


@pytest.mark.parametrize("want,kw", [
    (ERR_TYPE, dict(out_type=8)), (ERR_SHAPE, dict(head_dim=96)), (ERR_SHAPE, dict(n_heads=9)),
    (ERR_SHAPE, dict(n_kv_heads=0)), (ERR_SHAPE, dict(n_tok=-1)), (ERR_SHAPE, dict(scale=float("nan"))),
    (ERR_SHAPE, dict(q_stride=1016)), (ERR_SHAPE, dict(k_stride=260)), (ERR_SHAPE, dict(v_stride=0)),
    (ERR_NULL, dict(q=None)), (ERR_NULL, dict(v=None)), (ERR_NULL, dict(offsets=None)), (ERR_NULL, dict(out=None)),
    (ERR_ALIGN, dict(k=MIS)), (ERR_ALIGN, dict(out=MIS)), (ERR_ALIGN, dict(offsets=C + 2)), (OK, dict(n_tok=0)),
    (OK, dict(n_seq=0)),
])
def test_prompt_refusals(L, want, kw):
    a = {**PROMPT, **kw}
    assert L.qattn_prompt(*a.values(), None) == want


def test_binding_wants_cuda_tensors(L):
    x, i = torch.zeros(2, 8, 128), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        qg.KVCache(8, 128, 16, torch.zeros(16 * 8 * 144, dtype=torch.uint8))
    with pytest.raises(ValueError):
        qg.KVCache.empty(2, 8, 100)
    for call in (lambda: qg.kv_append(None, x, x, i), lambda: qg.kv_read(None, i), lambda: qg.kv_attend(None, x, i, i),
                 lambda: qg.prompt_attend(x, x, x, i)):
        with pytest.raises(TypeError):
            call()


def test_pages_of_a_cache(L):
    """Each reason for a refusal is named."""
    page = 8 * 16 * 144
    assert at._pages(0, 8, 128, 16) == 0 and at._pages(5 * page, 8, 128, 16) == 5
    most = (2 ** 31 - 1) // 16
    assert at._pages(most * 16 * 72, 1, 64, 16) == most
    for args, word in (((5 * page, 8, 96, 16), "heads of 64 or 128"), ((5 * page, 8, 128, 24), "multiple of 16"),
                       ((5 * page + 1, 8, 128, 16), "not a number of pages"),
                       (((most + 1) * 16 * 72, 1, 64, 16), "a cache has at most")):
        with pytest.raises(ValueError, match=word):
            at._pages(*args)


def test_rope_table():
    t = qg.rope_table(9, 8, base=100.0, device="cpu")
    assert t.shape == (9, 4, 2) and t.dtype == torch.float32
    assert abs(float(t[5, 1, 0]) - np.cos(5 * 100 ** -0.25)) < 1e-7 and float(t[0, 3, 1]) == 0.0
