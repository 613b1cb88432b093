"""GPU chunk attention (tq3_attention_chunk) where one call's queries, keys or values differ by many powers
of two: a row's result does not suffer by its neighbours' size, whichever kernel serves it.

The tolerance is that of test_gpu_tq3_chunk.py, with u = 2^-25 (half the spacing of subnormal fp16) added
where an operand is scaled by a factor that it shares:
* the logit. The largest |q~| of a row is 2^7 at least, so a coordinate is off by 2^-32 of it; with |q~_i| <=
  sqrt(128) |q|, |c|_1 <= sqrt(128) |c|_2 and the definition's post = 128^-1/2 that is
  2^-32 sqrt(128) scale |q| |k_j| < 2^-28 scale |q| |k_j|. A tile's keys share a factor that brings the largest
  f_j to 2^13 at least: u of that is 2^-38 f_max a coordinate, |q~|_1 <= 128 |q|, f_max <= |k|max / 1.276 (128
  centroids of 0.1129 at least), so 2^-38 sqrt(128) / 1.276 < 2^-34 scale |q| |k|max.
* a weight. The largest weight of a row is 2^6 at least, so one is off by 2^-31 of it (in the kernel for few
  rows a weight holds its value's factor: 2^-31 of the largest p f_v, times |c|_2 <= 0.9816 sqrt(128)).
* a value, 2^-38 of the largest f_v a coordinate: 2^-38 sqrt(128) / 1.276 < 2^-34 |v|max.
"""
import numpy as np
import pytest
import torch

from test_gpu_tq3_chunk import BF16, F32, H, POST, ROOM, Cache, to_np, wq  # noqa: F401 (wq is the fixture)
from weight_quantization_b200 import inputs

pytestmark = pytest.mark.gpu


def check(out, q, cache, new, bits, wide, scale):
    """Every row of every sequence within the bound."""
    signs = 2.0 * bits - 1.0
    group = q.shape[1] // cache.heads
    at = 0
    for b, n in enumerate(new):
        L = cache.keys[b]
        seen = np.arange(L) <= np.arange(L - n, L)[:, None]
        for h in range(cache.heads):
            f, c, _ = cache.dense(0, b, h, L)
            fv, cv, _ = cache.dense(1, b, h, L)
            kn, v = f * np.linalg.norm(c, axis=1), fv[:, None] * POST * (cv @ H) * signs
            vn = np.linalg.norm(v, axis=1)
            for g in range(group):
                x = q[at:at + n, h * group + g].astype(np.float64)
                qr, qn = (x * signs) @ H, np.linalg.norm(x, axis=1)[:, None]
                s = np.where(seen, scale * POST * (qr @ c.T) * f, -np.inf)
                p = np.exp(s - s.max(1, keepdims=True))
                largest = p.max(1) / p.sum(1)
                p /= p.sum(1, keepdims=True)
                ref = p @ v
                lam, w = (2.0 ** -20 + 24 * 2.0 ** -22, 2.0 ** -20) if wide else (2.0 ** -10 + 2.0 ** -15,) * 2
                ds = lam * scale * POST * (np.abs(qr) @ np.abs(c).T) * f
                ds += scale * qn * (2.0 ** -28 * kn + 2.0 ** -34 * kn.max())
                dist = np.linalg.norm(v[None] - ref[:, None], axis=2)
                bound = 1.05 * ((p * np.where(seen, ds, 0) * dist).sum(1) + w * (p @ vn))
                bound += (seen.sum(1) * (3 if wide else 1) / 16 + 32) * 2.0 ** -22 * (p @ vn)
                bound += 2.0 ** -34 * vn.max() + 2.0 ** -31 * (seen * np.maximum(
                    largest[:, None] * vn, (p * fv).max(1)[:, None] * 0.9816 * 128 ** 0.5)).sum(1)
                bound += (2.0 ** -24 if out.dtype == np.float32 else 2.0 ** -8) * np.linalg.norm(ref, axis=1)
                err = np.linalg.norm(out[at:at + n, h * group + g].astype(np.float64) - ref, axis=1)
                bad = ~(err <= bound)
                assert not bad.any(), (b, h, g, np.flatnonzero(bad)[:8], err[bad][:8], bound[bad][:8])
        at += n


def attend(wq, cache, q, new, room=ROOM, scale=128 ** -0.5):  # noqa: F811
    bits = inputs.tq3_sign_bits()
    pools, table = cache.device(room)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    kv = torch.tensor(cache.keys, dtype=torch.int32, device="cuda")
    out = wq.tq3_attention_chunk(q, *pools, table, start, kv, wq.sign_mask_words(bits), softmax_scale=scale)
    check(to_np(out), q.float().cpu().numpy(), cache, new, bits, q.dtype == F32, scale)
    assert wq.device_fault() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [-40, -24, 24, 28, 34, 40, 60])
@pytest.mark.parametrize("new,group,room", [([1], 8, ROOM), ([1, 1], 4, ROOM), ([20], 4, 0), ([60], 4, ROOM)])
def test_one_query_row_of_another_size(wq, new, group, room, power, dtype):  # noqa: F811
    """One row is 2^power times the others of its block of eight: heads of one KV head, tokens of a chunk."""
    cache = Cache([200, 90][:len(new)], 1, 16, seed=21)
    q = torch.from_numpy(inputs.gaussian((sum(new), group, 128), seed=5) * 2.0).to(dtype).cuda()
    q[sum(new) // 3, group // 2] *= 2.0 ** power
    attend(wq, cache, q, new, room)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [12, 20, 24])
@pytest.mark.parametrize("which", ["keys", "values", "both"])
@pytest.mark.parametrize("new,room", [(1, ROOM), (90, ROOM), (20, 0)])
def test_neighbours_of_another_size(wq, new, room, which, power, dtype):  # noqa: F811
    """A few keys or values are 2^power times their neighbours in a tile of 128. Rows before the last tokens do
    not see those; a key that all rows see takes all of a row's weight or none."""
    cache = Cache([300], 1, 16, seed=22)
    for pool, name, where in zip(cache.pools, ("keys", "values"), ([37, 297, 299], [296, 299])):
        for j in where if which in (name, "both") else ():
            pool[cache.table[0, j // 16], 0, j % 16, 48:].view(np.float32)[0] *= 2.0 ** power
    q = torch.from_numpy(inputs.gaussian((new, 4, 128), seed=6) * 3.0).to(dtype).cuda()
    attend(wq, cache, q, [new], room)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("grow", [8.0, -8.0])
@pytest.mark.parametrize("new", [1, 90])
def test_keys_that_grow_and_shrink(wq, new, grow, dtype):  # noqa: F811
    """Keys whose norms change by e^grow along the sequence, and by as much between neighbours for one in five."""
    n = 1100
    cache = Cache([n], 1, 16, seed=23)
    r = np.random.RandomState(24)
    for j in range(n):
        f = cache.pools[0][cache.table[0, j // 16], 0, j % 16, 48:].view(np.float32)
        f[0] *= np.exp(grow * (j / n - 0.5) + (r.uniform(-grow, grow) / 2 if j % 5 == 0 else 0.0))
    q = torch.from_numpy(inputs.gaussian((new, 4, 128), seed=7) * 0.1).to(dtype).cuda()
    attend(wq, cache, q, [new])
