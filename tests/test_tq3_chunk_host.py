"""Host-side refusals of tq3_attention_chunk (no GPU needed): the status codes that include/wq.h
documents, before anything is enqueued, and the binding's own checks."""
import math

import numpy as np
import pytest
import torch

from weight_quantization_b200 import ops

OK, NULL, SHAPE, DTYPE, ALIGN = 0, -1, -2, -3, -4
A = 0x10000  # an aligned fake device address: the checks fail before any use
M = np.zeros(4, np.uint32)


@pytest.fixture(scope="module")
def lib():
    from weight_quantization_b200 import build
    build.build()
    return ops.lib()


ARGS = dict(q=A, dtype=1, tokens=4, q_heads=8, qt=1024, qh=128, kp=A, vp=A, pages=3, heads=2, page=16, table=A, batch=2,
            pps=3, start=A, kv=A, max_q=4, window=0, sinks=0, mask=M.ctypes.data, scale=0.1, out=A, odtype=1, ws=A,
            ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=0), OK), (dict(batch=0), OK), (dict(batch=0, q=None, ws=None), OK), (dict(tokens=-1), SHAPE),
    (dict(tokens=1 << 31), SHAPE), (dict(tokens=1 << 30), SHAPE), (dict(batch=-1), SHAPE), (dict(pps=-1), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=3), SHAPE), (dict(q_heads=1), SHAPE), (dict(q_heads=0), SHAPE),
    (dict(page=12), SHAPE), (dict(max_q=-1), SHAPE), (dict(window=-1), SHAPE), (dict(window=1 << 31), SHAPE),
    (dict(sinks=-1), SHAPE), (dict(sinks=1 << 31), SHAPE), (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE),
    (dict(qt=-1024), SHAPE), (dict(qh=1 << 50), SHAPE), (dict(ws_bytes=1000), SHAPE), (dict(dtype=2), DTYPE),
    (dict(odtype=-1), DTYPE), (dict(q=None), NULL), (dict(kp=None), NULL), (dict(vp=None), NULL), (dict(table=None), NULL),
    (dict(start=None), NULL), (dict(kv=None), NULL), (dict(mask=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
    (dict(q=A + 8), ALIGN), (dict(kp=A + 8), ALIGN), (dict(vp=A + 4), ALIGN), (dict(table=A + 2), ALIGN),
    (dict(start=A + 2), ALIGN), (dict(kv=A + 1), ALIGN), (dict(out=A + 8), ALIGN), (dict(ws=A + 8), ALIGN),
    (dict(qt=1028), ALIGN), (dict(qh=132), ALIGN)])
def test_refusals(lib, change, status):
    assert lib.tq3_attention_chunk(*dict(ARGS, **change).values()) == status


def test_workspace(lib):
    assert lib.tq3_attention_chunk_workspace(-1, 4) == -1
    assert lib.tq3_attention_chunk_workspace(1, 0) == -1
    for max_q, group in ((0, 1), (1, 8), (4096, 8), (1 << 31, 1 << 31)):
        assert 0 < lib.tq3_attention_chunk_workspace(max_q, group) < 1 << 30


def test_binding_refuses_host_tensors():
    q = torch.zeros((4, 2, 128))
    pool = torch.zeros((1, 2, 16, 56), dtype=torch.uint8)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.tq3_attention_chunk(q, pool, pool, i[None], i, i[:1], M)
