"""GPU attention of ragged chunks over a paged TQ3 cache (tq3_attention_chunk) against its definition in
64 bits, on records of random indices, norms and scales.

Tolerances, derived from the operands' roundings (u the half step of a type). A logit is
    s_ij = scale f_j post (q~_i . c[idx_j])        (q~ = H (signs . q), f_j = norm_j scale_j)
and its abs sum A_ij = scale f_j post (|q~_i| . |c[idx_j]|). Where q and out are bf16 the operands are
fp16: q~ is rounded by 2^-11, the centroids by 1.4e-5 or, times the key's factor, by 2^-11, and the fp32
accumulations, the transform's 7 roundings and a few of the factors stay below 2^-16 together:
|ds_ij| <= L A_ij with L = 2^-10 + 2^-15. A weight is off by that, by its own rounding, 2^-11, and the
value's operand by another 2^-11 (or 1.4e-5), exp2 and log2 by 2^-21; the denominator has ds_ij alone. So
to first order
    |out_i - exact| <= sum_j p_ij |ds_ij| |v_j - out_i| + sum_j p_ij (2^-10 + 2^-15) |v_j|
in the 2-norm, to which 5% is added for the second order, and the bf16 result's 2^-8 |out_i|. Accumulating
the values, n_i of them, costs at most (n_i / 16 + 32) 2^-22 sum_j p_ij |v_j|, a tensor-core accumulation
taken as 2^-22. With fp32 on either side an operand is hi + lo, two roundings of 2^-11 (2^-22), the
dropped lo lo another 2^-22: L = 2^-20 + 24 accumulations of 2^-22, and 2^-20 in place of 2^-10 + 2^-15.
"""
import numpy as np
import pytest
import torch

from weight_quantization_b200 import inputs

pytestmark = pytest.mark.gpu

H = np.array([[1.0 - 2.0 * (bin(i & j).count("1") & 1) for j in range(128)] for i in range(128)])
CENTROIDS = np.array([-0.9816, -0.6168, -0.3479, -0.1129, 0.1129, 0.3479, 0.6168, 0.9816], np.float32).astype(np.float64)
POST = 128.0 ** -0.5
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def wq():
    from weight_quantization_b200 import build, ops
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ops.device_fault()
    return ops


ROOM = 240000  # keys that a test's table has room for: with less, few rows choose the kernel for few rows


def widened(table, page_size, room=ROOM):
    """The table on the device, its rows widened by entries that no token needs."""
    more = max(0, room // page_size - table.shape[1])
    return torch.from_numpy(np.pad(table, ((0, 0), (0, more)), constant_values=-1)).cuda()


class Cache:
    """Pools of random records, one page table, on the host and on the device."""

    def __init__(self, keys, heads, page_size, seed=0, spare=2, scale=1.0):
        r = np.random.RandomState(seed)
        need = [-(-n // page_size) for n in keys]
        self.keys, self.heads, self.page_size = keys, heads, page_size
        self.pages = sum(need) + spare
        self.pools = []
        for _ in range(2):
            p = r.randint(0, 256, (self.pages, heads, page_size, 56)).astype(np.uint8)
            f = np.empty(p.shape[:3] + (2,), np.float32)
            f[..., 0], f[..., 1] = r.uniform(3.0, 12.0, f.shape[:3]) * scale, r.uniform(0.15, 0.3, f.shape[:3])
            p[..., 48:] = f.view(np.uint8).reshape(p.shape[:3] + (8,))
            self.pools.append(p)
        order = r.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(keys), max(need + [0]) + 1), -1, np.int32)
        for b, n in enumerate(need):
            self.table[b, :n], order = order[:n], order[n:]

    def device(self, room=ROOM):
        return [torch.from_numpy(p).cuda() for p in self.pools], widened(self.table, self.page_size, room)

    def dense(self, which, b, h, n):
        """(norm * scale, centroids [n, 128]) of keys 0 .. n - 1; zeros without a page, and which have one."""
        j = np.arange(n)
        page = self.table[b, j // self.page_size]
        ok = (page >= 0) & (page < self.pages)
        rec = self.pools[which][np.where(ok, page, 0), h, j % self.page_size]
        bits = np.unpackbits(rec[:, :48], axis=1, bitorder="little").reshape(n, 128, 3)
        f = np.ascontiguousarray(rec[:, 48:]).view(np.float32).astype(np.float64)
        return f[:, 0] * f[:, 1], CENTROIDS[bits[:, :, 0] + 2 * bits[:, :, 1] + 4 * bits[:, :, 2]], ok


def check(out, q, cache, new, bits, wide, window=0, sinks=0, scale=128 ** -0.5, first=0, keys=None):
    """Rows of every sequence within the bound; rows that see nothing exactly zero."""
    signs = 2.0 * bits - 1.0
    group = q.shape[1] // cache.heads
    keys = cache.keys if keys is None else keys
    at = first
    for b, n in enumerate(new):
        L = keys[b]
        pos = np.arange(L - n, L)
        j = np.arange(L)
        for h in range(cache.heads):
            f, c, ok = cache.dense(0, b, h, L)
            fv, cv, _ = cache.dense(1, b, h, L)
            seen = (j <= pos[:, None]) & ok
            if window:
                seen &= (j > pos[:, None] - window) | (j < sinks)
            v = fv[:, None] * POST * (cv @ H) * signs
            for g in range(group):
                qr = (q[at:at + n, h * group + g].astype(np.float64) * signs) @ H
                s = scale * POST * (qr @ c.T) * f
                A = scale * POST * (np.abs(qr) @ np.abs(c).T) * f
                s = np.where(seen, s, -np.inf)
                top = np.where(seen.any(1), s.max(1, initial=-np.inf), 0.0)
                p = np.exp(s - top[:, None])
                total = p.sum(1, keepdims=True)
                p = p / np.where(total == 0, 1.0, total)
                ref = p @ v
                got = out[at:at + n, h * group + g].astype(np.float64)
                vn = np.linalg.norm(v, axis=1)
                dist = np.linalg.norm(v[None] - ref[:, None], axis=2)
                lam = 2.0 ** -20 + 24 * 2.0 ** -22 if wide else 2.0 ** -10 + 2.0 ** -15
                w = 2.0 ** -20 if wide else 2.0 ** -10 + 2.0 ** -15
                count = seen.sum(1) * (3 if wide else 1)
                bound = 1.05 * ((p * lam * np.where(seen, A, 0) * dist).sum(1) + w * (p @ vn))
                bound += (count / 16 + 32) * 2.0 ** -22 * (p @ vn)
                half = 2.0 ** -8 if out.dtype != np.float32 else 2.0 ** -24
                bound += half * np.linalg.norm(ref, axis=1)
                err = np.linalg.norm(got - ref, axis=1)
                bad = ~(err <= bound)
                assert not bad.any(), (b, h, g, np.flatnonzero(bad)[:8], err[bad][:8], bound[bad][:8])
                assert np.all(got[~seen.any(1)] == 0)
        at += n


def to_np(t):
    """fp32 as it is, bf16 as float64: its type tells `check` which rounding to allow."""
    return t.cpu().numpy() if t.dtype == F32 else t.float().cpu().numpy().astype(np.float64)


def run(wq, cache, new, group, dtype=BF16, out_dtype=None, window=0, sinks=0, seed=1, q_scale=0.3, sign_seed=42, max_q=None, room=ROOM):
    bits = inputs.tq3_sign_bits(sign_seed)
    pools, table = cache.device(room)
    n = sum(new)
    q = torch.from_numpy(inputs.gaussian((n, cache.heads * group, 128), seed=seed) * q_scale).to(dtype).cuda()
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    kv = torch.tensor(cache.keys, dtype=torch.int32, device="cuda")
    out = wq.tq3_attention_chunk(q, *pools, table, start, kv, wq.sign_mask_words(bits), max_q=max_q, window=window,
                                 sinks=sinks, out_dtype=out_dtype)
    wide = dtype == F32 or out.dtype == F32
    check(to_np(out), q.float().cpu().numpy(), cache, new, bits, wide, window, sinks)
    assert wq.device_fault() == 0
    return out


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys,new,heads,group,page_size", [
    ([1], [1], 1, 1, 16), ([5, 128, 129, 17], [1, 1, 1, 1], 2, 4, 16), ([515], [1], 3, 8, 32), ([300], [1], 1, 7, 1),
    ([77, 40], [1, 3], 2, 2, 2), ([90, 200], [2, 5], 1, 4, 4), ([131], [9], 2, 1, 8), ([400, 64, 1], [33, 64, 1], 2, 2, 64),
    ([16, 0, 31], [16, 0, 4], 1, 8, 16), ([1000], [1], 1, 16, 16), ([256], [70], 1, 5, 256), ([260], [40], 2, 20, 128)])
def test_against_the_definition(wq, keys, new, heads, group, page_size, dtype):
    run(wq, Cache(keys, heads, page_size, seed=len(keys) + keys[0]), new, group, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (100, 0), (128, 64), (200, 300), (1000, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("new", [(1, 1, 1), (40, 1, 7)])
def test_window_and_sinks(wq, window, sinks, new, dtype):
    run(wq, Cache([700, 450, 9], 2, 16, seed=3), list(new), 4, dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_little_work_in_blocks_of_eight_rows(wq, window, sinks, dtype):
    """A narrow table: a chunk of many rows on the kernel for few."""
    run(wq, Cache([300, 77], 2, 16, seed=18), [60, 1], 4, dtype, window=window, sinks=sinks, room=0)


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F32, BF16)])
def test_types_and_another_sign_table(wq, dtype, out_dtype):
    run(wq, Cache([333, 20], 2, 8, seed=5), [5, 20], 3, dtype, out_dtype, sign_seed=7)


@pytest.mark.parametrize("max_q", [0, 1, 64])
def test_more_new_tokens_than_max_q(wq, max_q):
    run(wq, Cache([333, 200], 1, 16, seed=5), [150, 2], 4, max_q=max_q)


def test_tokens_that_see_nothing(wq):
    """More new tokens than keys: the first ones are before the sequence's start."""
    cache = Cache([3, 0, 1], 2, 16, seed=6)
    bits = inputs.tq3_sign_bits()
    pools, table = cache.device()
    q = torch.from_numpy(inputs.gaussian((15, 4, 128), seed=2)).cuda()
    start = torch.tensor([0, 8, 10, 15], dtype=torch.int32, device="cuda")
    out = torch.full((15, 4, 128), 5.0, device="cuda")
    wq.tq3_attention_chunk(q, *pools, table, start, torch.tensor(cache.keys, dtype=torch.int32, device="cuda"),
                           wq.sign_mask_words(bits), out=out)
    check(to_np(out), q.cpu().numpy(), cache, [8, 2, 5], bits, True)
    blind = [0, 1, 2, 3, 4, 8, 9, 10, 11, 12, 13]
    assert torch.all(out[blind] == 0) and torch.all(out[[5, 6, 7, 14]].abs().amax(-1) > 0)


def test_rows_of_no_sequence_and_strided_queries(wq):
    cache = Cache([100, 33], 2, 16, seed=7)
    bits = inputs.tq3_sign_bits()
    pools, table = cache.device()
    fused = torch.from_numpy(inputs.gaussian((50, 12, 128), seed=3)).cuda()
    for q in (fused[:, 4:8], fused.transpose(0, 1).contiguous().transpose(0, 1)[:, 1:5]):
        start = torch.tensor([6, 11, 44], dtype=torch.int32, device="cuda")
        out = torch.full((50, 4, 128), 9.0, device="cuda")
        wq.tq3_attention_chunk(q, *pools, table, start, torch.tensor(cache.keys, dtype=torch.int32, device="cuda"),
                               wq.sign_mask_words(bits), out=out)
        assert torch.all(out[:6] == 9.0) and torch.all(out[44:] == 9.0)
        check(to_np(out), q.cpu().numpy(), cache, [5, 33], bits, True, first=6)


@pytest.mark.parametrize("page_size", [1, 8, 16, 64])
@pytest.mark.parametrize("new", [1, 60])
def test_pages_outside_the_pool_and_freed_pages(wq, page_size, new):
    """A hole in the table is masked out and reported; pages behind the window may be gone."""
    bits = inputs.tq3_sign_bits()
    cache = Cache([320], 2, page_size, seed=8)
    cache.table[0, 130 // page_size] = cache.pages
    cache.table[0, 200 // page_size] = -3
    pools, table = cache.device()
    q = torch.from_numpy(inputs.gaussian((new, 4, 128), seed=4) * 0.3).cuda()
    start = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    kv = torch.tensor([320], dtype=torch.int32, device="cuda")
    m = wq.sign_mask_words(bits)
    out = wq.tq3_attention_chunk(q, *pools, table, start, kv, m)
    assert wq.device_fault() == 64
    check(to_np(out), q.cpu().numpy(), cache, [new], bits, True)
    # keys that a window of 32 with 5 sinks leaves to the first row: 5 and from 320 - new + 1 - 32 on
    cache = Cache([320], 2, page_size, seed=9)
    low = 320 - new + 1 - 32
    for p in range(cache.table.shape[1] - 1):
        if p * page_size >= 5 and (p + 1) * page_size <= low:
            cache.table[0, p] = -1
    pools, table = cache.device()
    out = wq.tq3_attention_chunk(q, *pools, table, start, kv, m, window=32, sinks=5)
    assert wq.device_fault() == 0
    check(to_np(out), q.cpu().numpy(), cache, [new], bits, True, window=32, sinks=5)


def test_more_keys_than_the_table_holds(wq):
    """kv_len beyond the table counts as the table's keys, and is reported."""
    bits = inputs.tq3_sign_bits()
    cache = Cache([64], 1, 16, seed=10)
    pools, table = cache.device()
    table = table[:, :4].contiguous()
    q = torch.from_numpy(inputs.gaussian((3, 2, 128), seed=4)).cuda()
    out = wq.tq3_attention_chunk(q, *pools, table, torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                                 torch.tensor([100], dtype=torch.int32, device="cuda"), wq.sign_mask_words(bits))
    assert wq.device_fault() == 64
    check(to_np(out), q.cpu().numpy(), cache, [3], bits, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 50])
def test_nan_and_infinities_in_masked_places(wq, new, dtype):
    """Records behind kv_len, of the future and of the window's past hold NaN and infinite factors; a NaN
    query spoils only its own row."""
    bits = inputs.tq3_sign_bits()
    n = 150 - new  # the last sequence's tokens all see keys 0 .. n at least
    cache = Cache([160], 1, 16, seed=11)
    clean = [p.copy() for p in cache.pools]
    bad = np.array([np.nan, np.inf], np.float32).view(np.uint8)
    for p in cache.pools:
        for j in list(range(150, 160)) + list(range(8, 20)):
            p[cache.table[0, j // 16], 0, j % 16, 48:] = bad
    pools, table = cache.device()
    cache.pools = clean
    q = torch.from_numpy(inputs.gaussian((new, 4, 128), seed=4) * 0.3).to(dtype).cuda()
    if new > 1:
        q[2, 1, 77] = float("nan")
        q[3, 2, 5] = float("inf")
    out = wq.tq3_attention_chunk(q, *pools, table, torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                                 torch.tensor([150], dtype=torch.int32, device="cuda"), wq.sign_mask_words(bits),
                                 window=60, sinks=8)
    x, y = to_np(out), q.float().cpu().numpy()
    if new > 1:
        assert np.isnan(x[2, 1]).all() and np.isnan(x[3, 2]).all()
        assert np.isnan(x).reshape(-1, 128).any(1).sum() == 2
        y[2, 1], y[3, 2] = y[2, 0], y[3, 1]
        x[2, 1], x[3, 2] = x[2, 0], x[3, 1]  # their places are checked above
    check(x, y, cache, [new], bits, dtype == F32, window=60, sinks=8, keys=[150])


@pytest.mark.parametrize("new", [1, 48])
@pytest.mark.parametrize("q_scale,kv_scale", [(1e-20, 1.0), (1.0, 1e-12), (1e4, 1e-4), (1.0, 1e12), (1e-30, 1e30)])
def test_magnitudes(wq, q_scale, kv_scale, new):
    """The operands' range does not depend on the data's: logits near 1, or all equal, on tiny and huge
    queries, keys and values."""
    bits = inputs.tq3_sign_bits()
    cache = Cache([200], 2, 16, seed=12, scale=kv_scale)
    pools, table = cache.device()
    q = torch.from_numpy(inputs.gaussian((new, 2, 128), seed=4).astype(np.float64) * q_scale).float().cuda()
    scale = 128 ** -0.5 / max(q_scale * kv_scale, 1e-30) if q_scale * kv_scale > 1 else 128 ** -0.5
    out = wq.tq3_attention_chunk(q, *pools, table, torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                                 torch.tensor([200], dtype=torch.int32, device="cuda"), wq.sign_mask_words(bits),
                                 softmax_scale=scale)
    check(to_np(out), q.cpu().numpy(), cache, [new], bits, True, scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("keys_grow,values_grow", [(2.0, 8.0), (-2.0, -8.0), (0.0, 12.0)])
def test_norms_that_grow_and_shrink(wq, new, dtype, keys_grow, values_grow):
    """Factors that change by e^grow along the sequence, and by as much between neighbours for one key in
    five: running maxima are raised, and values of very different length share a tile."""
    bits = inputs.tq3_sign_bits()
    n = 1100
    cache = Cache([n], 1, 16, seed=15)
    r = np.random.RandomState(16)
    for pool, grow in zip(cache.pools, (keys_grow, values_grow)):
        for j in range(n):
            f = pool[cache.table[0, j // 16], 0, j % 16, 48:].view(np.float32)
            f[0] *= np.exp(grow * (j / n - 0.5) + (r.uniform(-grow, grow) / 2 if j % 5 == 0 else 0.0))
    pools, table = cache.device()
    q = torch.from_numpy(inputs.gaussian((new, 4, 128), seed=4)).to(dtype).cuda()
    out = wq.tq3_attention_chunk(q, *pools, table, torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                                 torch.tensor([n], dtype=torch.int32, device="cuda"), wq.sign_mask_words(bits))
    check(to_np(out), q.float().cpu().numpy(), cache, [new], bits, dtype == F32)
    assert wq.device_fault() == 0


def test_two_streams_at_once(wq):
    """Calls of both kernels on two streams, interleaved, give what each gives alone."""
    bits = inputs.tq3_sign_bits()
    m = wq.sign_mask_words(bits)
    cache = Cache([900, 300, 700, 1200], 2, 16, seed=17)
    pools, table = cache.device()
    kv = torch.tensor(cache.keys, dtype=torch.int32, device="cuda")
    new = [1, 70, 1, 200]
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    qs = [torch.from_numpy(inputs.gaussian((sum(new), 8, 128), seed=s) * 0.3).to(BF16).cuda() for s in (1, 2)]
    alone = [wq.tq3_attention_chunk(q, *pools, table, start, kv, m) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(wq.tq3_attention_chunk(qs[i], *pools, table, start, kv, m))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


@pytest.mark.parametrize("new", [1, 130])
def test_same_bits_every_time_and_captured(wq, new):
    """Two runs give the same bits; so does a captured graph on a stream of its own, replayed on new
    inputs and lengths in the same buffers."""
    bits = inputs.tq3_sign_bits()
    m = wq.sign_mask_words(bits)
    cache = Cache([900, 300, 700], 2, 16, seed=13)
    pools, table = cache.device()
    q = torch.empty((3 * new, 8, 128), dtype=BF16, device="cuda")
    start = torch.tensor([0, new, 2 * new, 3 * new], dtype=torch.int32, device="cuda")
    kv = torch.tensor([900, 300, 700], dtype=torch.int32, device="cuda")
    q.copy_(torch.from_numpy(inputs.gaussian(tuple(q.shape), seed=1) * 0.3))
    a = wq.tq3_attention_chunk(q, *pools, table, start, kv, m, max_q=new)
    b = wq.tq3_attention_chunk(q, *pools, table, start, kv, m, max_q=new)
    assert torch.equal(a, b)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out, other = torch.empty_like(q), torch.empty_like(q)
    with torch.cuda.stream(stream):
        wq.tq3_attention_chunk(q, *pools, table, start, kv, m, max_q=new, out=out)
    stream.synchronize()
    assert torch.equal(a, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        wq.tq3_attention_chunk(q, *pools, table, start, kv, m, max_q=new, out=out)
        wq.tq3_attention_chunk(q, *pools, table, start, kv, m, max_q=new, window=64, sinks=2, out=other)
    for seed, lengths in ((2, [900, 290, 131]), (3, [850, 150, 700])):
        q.copy_(torch.from_numpy(inputs.gaussian(tuple(q.shape), seed=seed) * 0.3))
        kv.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        x = q.float().cpu().numpy()
        check(to_np(out), x, cache, [new] * 3, bits, False, keys=lengths)
        check(to_np(other), x, cache, [new] * 3, bits, False, window=64, sinks=2, keys=lengths)
    assert wq.device_fault() == 0


def test_offsets_past_32_bits(wq):
    """Pages that lie beyond the first 4 GiB of their pool."""
    bits = inputs.tq3_sign_bits()
    page_size, heads = 128, 2
    small = Cache([300, 140], heads, page_size, seed=14, spare=0)
    pages = (1 << 32) // (heads * page_size * 56) + 5 + small.pages
    pools = [torch.zeros((pages, heads, page_size, 56), dtype=torch.uint8, device="cuda") for _ in range(2)]
    shift = pages - small.pages
    for p, x in zip(pools, small.pools):
        p[shift:] = torch.from_numpy(x).cuda()
    table = np.where(small.table >= 0, small.table + shift, -1).astype(np.int32)
    for new in ([1, 1], [100, 3]):
        q = torch.from_numpy(inputs.gaussian((sum(new), 8, 128), seed=4) * 0.3).cuda()
        start = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
        out = wq.tq3_attention_chunk(q, *pools, widened(table, page_size), start,
                                     torch.tensor([300, 140], dtype=torch.int32, device="cuda"),
                                     wq.sign_mask_words(bits))
        check(to_np(out), q.cpu().numpy(), small, new, bits, True)
    assert wq.device_fault() == 0


def test_a_serving_run(wq):
    """Prompt chunks and single tokens appended, attended to and read back, step by step, as a server
    does: each step's attention is over what the cache then decodes to."""
    bits = inputs.tq3_sign_bits()
    m = wq.sign_mask_words(bits)
    heads, group, page_size, width = 2, 4, 16, 12
    pools = [torch.zeros((30, heads, page_size, 56), dtype=torch.uint8, device="cuda") for _ in range(2)]
    order = torch.randperm(30, generator=torch.Generator().manual_seed(1))[:2 * width]
    cache = Cache([0, 0], heads, page_size)
    cache.pages, cache.table = 30, order.view(2, width).to(torch.int32).numpy()
    table = widened(cache.table, page_size)
    lengths = [0, 0]
    for step, new in enumerate([(70, 5), (1, 60), (1, 1), (30, 1), (1, 1)]):
        n = sum(new)
        fused = torch.from_numpy(inputs.gaussian((n, heads * (group + 2), 128), seed=20 + step)).to(BF16).cuda()
        q, k, v = fused[:, :heads * group], fused[:, heads * group:-heads], fused[:, -heads:]
        slots = []
        for b in range(2):
            at = np.arange(lengths[b], lengths[b] + new[b])
            slots += (cache.table[b, at // page_size].astype(np.int64) * page_size + at % page_size).tolist()
            lengths[b] += new[b]
        wq.tq3_cache_append(k, v, m, torch.tensor(slots, device="cuda"), *pools)
        start = torch.tensor([0, new[0], n], dtype=torch.int32, device="cuda")
        kv = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        out = wq.tq3_attention_chunk(q, *pools, table, start, kv, m, max_q=max(new))
        cache.pools = [p.cpu().numpy() for p in pools]
        check(to_np(out), q.float().cpu().numpy(), cache, list(new), bits, False, keys=lengths)
        starts = torch.tensor([0, lengths[0], sum(lengths)], dtype=torch.int32, device="cuda")
        dense = wq.tq3_cache_read(*pools, table, starts, m, sum(lengths), out_dtype=F32)
        for i in range(2):
            f, c, _ = cache.dense(i, 0, 1, lengths[0])
            ref = f[:, None] * POST * (c @ H) * (2.0 * bits - 1.0)
            assert np.allclose(dense[i][:lengths[0], 1].cpu().numpy(), ref, rtol=0, atol=1e-5 * np.abs(ref).max())
    assert wq.device_fault() == 0
