"""Host-side refusals of the calls on a batch's paged cache (no GPU needed): the status codes that
include/wq.h documents, before anything is enqueued, and the binding's own checks."""
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


def call(fn, order, defaults, **change):
    a = dict(defaults, **change)
    return fn(*[a[n] for n in order])


APPEND = dict(k=A, v=A, dtype=1, tokens=4, heads=2, kt=256, kh=128, vt=256, vh=128, mask=M.ctypes.data, slots=A, kp=A,
              vp=A, pages=3, page=16, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=0), OK), (dict(tokens=0, k=None, kp=None), OK), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 41), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE), (dict(pages=-1), SHAPE), (dict(page=0), SHAPE),
    (dict(page=24), SHAPE), (dict(page=1 << 31), SHAPE), (dict(pages=1 << 50, page=1 << 20), SHAPE),
    (dict(kt=-256), SHAPE), (dict(vh=1 << 50), SHAPE), (dict(dtype=2), DTYPE), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(mask=None), NULL), (dict(slots=None), NULL), (dict(kp=None), NULL), (dict(vp=None), NULL),
    (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(slots=A + 4), ALIGN), (dict(kp=A + 8), ALIGN),
    (dict(kt=260), ALIGN), (dict(vh=132), ALIGN)])
def test_append_refusals(lib, change, status):
    assert call(lib.tq3_cache_append, list(APPEND), APPEND, **change) == status


READ = dict(kp=A, vp=A, pages=3, heads=2, page=16, table=A, batch=2, pps=3, start=A, tokens=9, mask=M.ctypes.data, ko=A,
            vo=A, dtype=1, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=0), OK), (dict(batch=0), OK), (dict(batch=0, kp=None, table=None), OK), (dict(tokens=-1), SHAPE),
    (dict(tokens=1 << 31), SHAPE), (dict(batch=-1), SHAPE), (dict(pps=-1), SHAPE), (dict(heads=0), SHAPE),
    (dict(page=3), SHAPE), (dict(dtype=9), DTYPE), (dict(kp=None), NULL), (dict(table=None), NULL),
    (dict(start=None), NULL), (dict(ko=None), NULL), (dict(mask=None), NULL), (dict(kp=A + 8), ALIGN),
    (dict(table=A + 2), ALIGN), (dict(start=A + 1), ALIGN), (dict(vo=A + 8), ALIGN)])
def test_read_refusals(lib, change, status):
    assert call(lib.tq3_cache_read, list(READ), READ, **change) == status


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 2, 128))
    pool = torch.zeros((1, 2, 16, 56), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.tq3_cache_append(x, x, M, torch.zeros(4, dtype=torch.int64), pool, pool)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.tq3_cache_read(pool, pool, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), M, 4)
