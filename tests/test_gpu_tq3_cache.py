"""GPU paged cache of a batch (tq3_cache_append, tq3_cache_read) against its definition in 64 bits.

append: the indices are those of real arithmetic, so they equal the fp64 restatement below exactly, on
ordinary vectors and at the exact ties (a coefficient of exactly 0 is the one tie that vectors of
floats reach: the fp64 sums below are exact on them). Norms and scales of vectors that stay on the fast
path, with u = 2^-24 and first-order bounds: the sum of 128 squares has chains of at most 16 fused adds
and three more, 20 roundings, halved by the square root, and one for the root: 11 u < 1e-6. The scale
adds the transform's error, at most 7 sqrt(128) u |x| <= 79 u of max|z|, the norm's 11 u and three
roundings: 93 u < 6e-6.

read: the bits of tq3_decode_paged on the same records (the oracle's decode, which that call is tested
against).
"""
import numpy as np
import pytest
import torch

from weight_quantization_b200 import inputs

pytestmark = pytest.mark.gpu

H = np.array([[1.0 - 2.0 * (bin(i & j).count("1") & 1) for j in range(128)] for i in range(128)])
BOUND = np.array([-0.7992, -0.4824, -0.2304, 0.0, 0.2304, 0.4824, 0.7992], np.float32).astype(np.float64)


@pytest.fixture(scope="module")
def wq():
    from weight_quantization_b200 import build, ops
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    ops.device_fault()
    return ops


def encode64(x, bits):
    """(indices, norms, scales) of rows of x in fp64."""
    x = x.astype(np.float64)
    z = (x * (2.0 * bits - 1.0)) @ H
    norm = np.maximum(np.sqrt((x * x).sum(1)), 1e-8)
    scale = np.maximum(np.abs(z).max(1) / (np.sqrt(128.0) * norm), 1e-8)
    over = norm > np.finfo(np.float32).max
    T = scale * np.sqrt(128.0) * norm
    idx = (z[:, :, None] > BOUND * T[:, None, None]).sum(2)
    idx[over], scale[over], norm[over] = 3, 1e-8, np.inf
    return idx, norm, scale


def unpack(records):
    b = np.unpackbits(records[:, :48], axis=1, bitorder="little").reshape(-1, 128, 3)
    return b[:, :, 0] + 2 * b[:, :, 1] + 4 * b[:, :, 2]


def check_records(rec, x, bits):
    idx, norm, scale = encode64(x, bits)
    assert np.array_equal(unpack(rec), idx)
    f = np.ascontiguousarray(rec[:, 48:]).view(np.float32).astype(np.float64)
    big = ~np.isfinite(norm)
    assert np.array_equal(f[big, 0], norm[big])
    assert np.all(np.abs(f[~big, 0] - norm[~big]) <= 1e-6 * norm[~big])
    assert np.all(np.abs(f[:, 1] - scale) <= 6e-6 * scale)


def append(wq, k, v, bits, page_size, seed=0, spare=2):
    """Append k and v [tokens, heads, 128] at random slots; returns (k records, v records) by token and
    the pools with the slots."""
    tokens, heads = k.shape[:2]
    pages = -(-tokens // page_size) + spare
    slots = torch.randperm(pages * page_size, generator=torch.Generator().manual_seed(seed))[:tokens].cuda()
    pools = [torch.full((pages, heads, page_size, 56), 7 + i, dtype=torch.uint8, device="cuda") for i in range(2)]
    wq.tq3_cache_append(k, v, wq.sign_mask_words(bits), slots, *pools)
    got = [p[slots // page_size, :, slots % page_size].cpu().numpy() for p in pools]
    touched = torch.zeros(pages * page_size, dtype=torch.bool, device="cuda")
    touched[slots] = True
    for i, p in enumerate(pools):  # records that no slot names keep their bytes
        assert torch.all(p.transpose(1, 2).reshape(-1, heads, 56)[~touched] == 7 + i)
    return got, pools, slots


@pytest.mark.parametrize("tokens,heads,page_size,dtype", [
    (1, 1, 16, torch.bfloat16), (1, 8, 1, torch.float32), (31, 3, 2, torch.bfloat16), (32, 2, 16, torch.float32),
    (33, 5, 8, torch.bfloat16), (257, 1, 64, torch.float32), (1000, 4, 16, torch.bfloat16),
    (130, 7, 256, torch.bfloat16)])
def test_append_matches_the_definition(wq, tokens, heads, page_size, dtype):
    bits = inputs.tq3_sign_bits()
    x = torch.from_numpy(inputs.gaussian((2, tokens, heads, 128), seed=tokens)).cuda()
    x[0, :, :, :4] *= 20
    x[1] += 2.0 * torch.from_numpy(inputs.gaussian((tokens, heads, 1), seed=3)).cuda()
    x = x.to(dtype)
    (rk, rv), _, _ = append(wq, x[0], x[1], bits, page_size)
    for rec, y in ((rk, x[0]), (rv, x[1])):
        check_records(rec.reshape(-1, 56), y.float().cpu().numpy().reshape(-1, 128), bits)
    assert wq.device_fault() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("seed", [42, 5])
def test_append_ties_and_extremes(wq, dtype, seed):
    """Constant and sparse vectors (coefficients of exactly 0), small integers, zeros, and magnitudes
    from the floors to the end of the fp32 range; the page's sign table and another."""
    bits = inputs.tq3_sign_bits(seed)
    r = np.random.RandomState(seed)
    rows = [np.full(128, c) for c in (1.0, -2.5, 1e-3)] + [np.eye(128)[i] * c for i, c in ((0, 1.0), (77, -3.0))]
    rows += [np.zeros(128), 2.0 * bits - 1.0, r.randint(-2, 3, 128), r.randint(0, 2, 128), np.tile([3.0, 0.0], 64)]
    g = r.randn(128)
    rows += [g * s for s in (1e-38, 1e-24, 3e-19, 1e-14, 1e-12, 1e-9, 1e-6, 1e6, 1e17, 1e19, 1e30, 1e37)]
    rows += [np.full(128, 3e38), np.eye(128)[5] * 2e38]
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(dtype).cuda()[:, None]
    (rk, rv), _, _ = append(wq, x, x.flip(0), bits, 16)
    y = x.float().cpu().numpy()[:, 0]
    check_records(rk[:, 0], y, bits)
    check_records(rv[:, 0], y[::-1], bits)


def test_append_near_ties(wq):
    """Vectors made so that a coefficient lies within 1e-7 of a boundary: fp32 alone decides some of
    them wrongly, the definition does not."""
    bits = inputs.tq3_sign_bits()
    r = np.random.RandomState(1)
    signs = 2.0 * bits - 1.0
    rows = []
    for n in range(400):
        z = r.uniform(-0.7, 0.7, 128)
        z[r.randint(128)] = 1.0 if n % 2 else -1.0
        z[r.randint(128)] = BOUND[n % 7] * (1 + r.uniform(-1e-7, 1e-7)) + (n % 7 == 3) * r.uniform(-1e-7, 1e-7)
        rows.append((H @ z) / 128 * signs)
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).cuda().view(200, 2, 128)
    (rk, rv), _, _ = append(wq, x, x, bits, 32)
    for rec in (rk, rv):
        check_records(rec.reshape(-1, 56), x.cpu().numpy().reshape(-1, 128), bits)


def test_append_slices_slots_and_faults(wq):
    """K and V as slices of a fused projection and as head-major tensors; negative slots are padding,
    slots outside the pool are skipped and reported."""
    bits = inputs.tq3_sign_bits()
    m = wq.sign_mask_words(bits)
    x = torch.from_numpy(inputs.gaussian((70, 10, 128), seed=8)).cuda().to(torch.bfloat16)
    k, v = x[:, 4:7], x.transpose(0, 1).contiguous().transpose(0, 1)[:, 7:10]
    (rk, rv), _, _ = append(wq, k, v, bits, 8)
    check_records(rk.reshape(-1, 56), k.float().cpu().numpy().reshape(-1, 128), bits)
    check_records(rv.reshape(-1, 56), v.float().cpu().numpy().reshape(-1, 128), bits)
    pools = [torch.zeros((4, 3, 8, 56), dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.full((70,), -1, dtype=torch.int64, device="cuda")
    slots[3], slots[69] = 31, 0
    wq.tq3_cache_append(k, v, m, slots, *pools)
    assert wq.device_fault() == 0
    for p, rec in zip(pools, (rk, rv)):
        assert np.array_equal(p[3, :, 7].cpu().numpy(), rec[3])
        assert np.array_equal(p[0, :, 0].cpu().numpy(), rec[69])
        assert int(p.count_nonzero()) == np.count_nonzero(rec[[3, 69]])
    slots[5], slots[6] = 32, 1 << 40
    before = [p.clone() for p in pools]
    wq.tq3_cache_append(k, v, m, slots, *pools)
    assert wq.device_fault() == 64
    assert all(torch.equal(a, b) for a, b in zip(before, pools))


@pytest.mark.parametrize("lengths,heads,page_size,dtype", [
    ([1], 1, 16, torch.float32), ([5, 0, 40], 2, 16, torch.bfloat16), ([0, 0, 33, 1, 64], 3, 1, torch.float32),
    ([100, 31, 0], 5, 2, torch.bfloat16), ([513, 2, 255], 4, 64, torch.bfloat16), ([7] * 90, 1, 8, torch.float32)])
def test_read_matches_the_paged_decoder(wq, lengths, heads, page_size, dtype):
    bits = inputs.tq3_sign_bits()
    m = wq.sign_mask_words(bits)
    r = np.random.RandomState(sum(lengths))
    need = [-(-n // page_size) for n in lengths]
    pages, width = sum(need) + 2, max(need) + 1
    pools = [torch.from_numpy(r.randint(0, 256, (pages, heads, page_size, 56), dtype=np.uint8)) for _ in range(2)]
    for p in pools:
        f = p.view(torch.float32)
        f[..., 12], f[..., 13] = torch.rand(f.shape[:-1]) * 9, torch.rand(f.shape[:-1])
    pools = [p.cuda() for p in pools]
    order = r.permutation(pages)
    table = np.full((len(lengths), width), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n], order = order[:n], order[n:]
    first = 3  # rows before the first sequence and after the last one stay
    start = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32) + first
    n_tokens = int(start[-1]) + 5
    outs = [torch.full((n_tokens, heads, 128), 9.0 + i, dtype=dtype, device="cuda") for i in range(2)]
    wq.tq3_cache_read(*pools, torch.from_numpy(table).cuda(), torch.from_numpy(start).cuda(), m, n_tokens,
                      k_out=outs[0], v_out=outs[1])
    assert wq.device_fault() == 0
    for i, (out, pool) in enumerate(zip(outs, pools)):
        assert torch.all(out[:first] == 9.0 + i) and torch.all(out[start[-1]:] == 9.0 + i)
        for b, n in enumerate(lengths):
            for h in range(heads):
                if n:
                    t = torch.from_numpy(table[b, :need[b]] * heads + h).cuda()
                    ref = wq.tq3_decode_paged(pool.view(-1, 56), t, page_size, n, m, out_dtype=dtype)
                    assert torch.equal(out[start[b]:start[b + 1], h], ref)


def test_read_outside_the_pool(wq):
    """A page outside the pool, and tokens past the table's width, decode as zeros and are reported."""
    m = wq.sign_mask_words(inputs.tq3_sign_bits())
    pools = [torch.full((3, 2, 4, 56), 0x3f, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = torch.tensor([[0, 3], [-5, 1]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 8, 18], dtype=torch.int32, device="cuda")
    k, v = wq.tq3_cache_read(*pools, table, start, m, 18, out_dtype=torch.float32)
    assert wq.device_fault() == 64
    dead = torch.tensor([False] * 4 + [True] * 4 + [True] * 4 + [False] * 4 + [True] * 2, device="cuda")
    for x in (k, v):
        assert torch.all(x[dead] == 0) and torch.all(x[~dead].abs().amax(-1) > 0)


def test_append_and_read_captured(wq):
    """Both calls in a CUDA graph on a stream of its own, replayed on new inputs in the same buffers."""
    bits = inputs.tq3_sign_bits()
    m = wq.sign_mask_words(bits)
    x = torch.empty((2, 48, 2, 128), dtype=torch.bfloat16, device="cuda")
    pools = [torch.zeros((4, 2, 16, 56), dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.randperm(64, device="cuda")[:48]
    slots = slots.sort().values
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    start = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    outs = [torch.empty((64, 2, 128), dtype=torch.float32, device="cuda") for _ in range(2)]
    stream = torch.cuda.Stream()

    def step():
        wq.tq3_cache_append(x[0], x[1], m, slots, *pools)
        wq.tq3_cache_read(*pools, table, start, m, 64, k_out=outs[0], v_out=outs[1])

    x.copy_(torch.from_numpy(inputs.gaussian(tuple(x.shape), seed=1)))
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for seed in (2, 3):
        x.copy_(torch.from_numpy(inputs.gaussian(tuple(x.shape), seed=seed)))
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            rec = pools[i].transpose(1, 2).reshape(64, 2, 56)[slots].cpu().numpy()
            check_records(rec.reshape(-1, 56), x[i].float().cpu().numpy().reshape(-1, 128), bits)
            # an encoded Gaussian vector is within cosine 0.9 of what it stands for
            back = outs[i][slots].reshape(-1, 128)
            cos = torch.nn.functional.cosine_similarity(back, x[i].float().reshape(-1, 128), dim=1)
            assert cos.min() > 0.9
