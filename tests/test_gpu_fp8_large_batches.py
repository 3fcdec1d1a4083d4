"""The 8-bit dispatch with eight vectors a thread, for each number of slots and with a
capacity, and the quantiser with four blocks a thread and a number of blocks that does not
fill the last: the forms that large batches take."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu
from oracle import fp8_oracle as X
from test_gpu_fp8 import f32, hard_rows, quantize_dev, u8

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("T,h,E,K,capacity", [
    (2501, 128, 4, 1, 0), (3001, 4096, 8, 2, 0), (2500, 4224, 16, 3, 0), (2600, 1152, 16, 4, 0), (3001, 4096, 128, 8, 0),
    (2500, 7168, 64, 6, 0), (2600, 384, 64, 16, 0), (2433, 8320, 32, 12, 0), (5003, 2048, 8, 2, 1100), (2999, 4096, 32, 8, 640)])
def test_permute_fp8(T, h, E, K, capacity):
    """Maps in ascending token order an expert, and under them the tokens' codes and scales."""
    M = lib()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert T * -(-h // 4096) >= 16 * sms                      # the rule of the eight-vector form
    rng = np.random.default_rng(T + h)
    idx = np.argsort(rng.random((T, E)) * np.linspace(1, 3, E), axis=1)[:, :K].astype(np.int32)
    prob = rng.random((T, K)).astype(np.float32)
    xq = torch.from_numpy(rng.integers(0, 256, (T, h), dtype=np.uint8)).cuda()
    xsf = torch.from_numpy(rng.random((T, h // 128)).astype(np.float32)).cuda()
    cfg = M.make_config(T, h, E, K, 128, capacity=capacity)
    ws = torch.empty(M.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets, dst = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T, K, **i32)
    src, pp = torch.full((T * K,), -9, **i32), f32(T * K)
    q, sf = u8(T * K, h), f32(T * K, h // 128)
    M.moe_permute_fp8(cfg, xq, xsf, torch.from_numpy(idx).cuda(), torch.from_numpy(prob).cuda(), q, sf, counts, offsets, dst,
                      src, pp, ws)
    assert M.moe_get_error() == M.MOE_OK
    order = np.argsort(idx.ravel(), kind="stable")
    total = np.bincount(idx.ravel(), minlength=E)
    first = np.concatenate([[0], np.cumsum(total)])
    keep = [order[first[e]:first[e + 1]][:capacity or None] for e in range(E)]
    pairs = np.concatenate(keep)
    kept = np.array([len(k) for k in keep])
    assert (len(pairs) < T * K) == (capacity > 0)
    want = np.full(T * K, -1)
    want[pairs] = np.arange(len(pairs))
    np.testing.assert_array_equal(dst.cpu().numpy().ravel(), want)
    np.testing.assert_array_equal(counts.cpu().numpy(), kept)
    np.testing.assert_array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(kept)]))
    n = len(pairs)
    np.testing.assert_array_equal(src.cpu().numpy()[:n], pairs // K)
    np.testing.assert_array_equal(pp.cpu().numpy()[:n], prob.ravel()[pairs])
    token = torch.from_numpy(pairs // K).cuda()
    assert torch.equal(q[:n], xq[token]) and torch.equal(sf[:n], xsf[token])
    assert torch.all(q[n:] == 0xEE) and torch.all(sf[n:] == 77.0) and torch.all(src[n:] == -9) and torch.all(pp[n:] == 77.0)


@pytest.mark.parametrize("rows,K", [(1393, 7296), (9001, 1152), (80001, 128)])
def test_quantize_bit_exact(rows, K):
    M = lib()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = rows * (K // 128)
    assert blocks >= 512 * sms and blocks % 128 != 0          # four blocks a thread, the last block of threads not full
    rng = np.random.default_rng(rows)
    x = hard_rows(rng, rows, K)
    x[-9:] = hard_rows(rng, 9, K)                             # (non-finite and subnormal blocks at the end too)
    pad = u8(rows * K + 256), f32(rows * (K // 128) + 64)
    q, sf = quantize_dev(M, x)
    q2, sf2 = pad[0][:rows * K].view(rows, K), pad[1][:blocks].view(rows, K // 128)
    M.moe_fp8_quantize(rows, K, torch.from_numpy(x).bfloat16().cuda(), q2, sf2)
    oq, osf = X.quantize(x)
    np.testing.assert_array_equal(sf.cpu().numpy(), osf)
    np.testing.assert_array_equal(q.cpu().numpy(), oq)
    assert torch.equal(q2, q) and torch.equal(sf2.view(torch.int32), sf.view(torch.int32))
    assert torch.all(pad[0][rows * K:] == 0xEE) and torch.all(pad[1][blocks:] == 77.0)
