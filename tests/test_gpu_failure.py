"""The bounded-wait failure path on the GPU, without a fault: a self-test kernel built from the
GEMM kernels' wait helpers waits on a barrier that nothing arrives on, gives up after a short
limit, records FP8Q_ERR_TIMEOUT in the device error word, stops its other warps through the abort
flag and releases TMEM.  The host reads the status, and the next kernels run correctly on the same
context."""
import time

import numpy as np
import pytest
import torch

import oracle
import fp8_blockwise_w8a8_b200 as fq
from fp8_blockwise_w8a8_b200 import inputs

from helpers import dev_bf16, dev_f32, dev_u8, host_bf16_f64, assert_within_gemm_tolerance, promoted_steps

pytestmark = pytest.mark.gpu


def test_timeout_is_reported_and_the_context_stays_usable():
    assert fq.check_device_error() == 0
    t0 = time.perf_counter()
    fq.selftest_timeout(2_000_000)                       # 2 ms
    assert fq.check_device_error() == fq.FP8Q_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 5.0
    assert fq.check_device_error() == 0                  # the word was cleared by the read
    # the same context quantizes and multiplies correctly afterwards
    d = inputs.tiny_linear()
    aq, sa = oracle.quant_token_1x128(d["A"])
    wq, sw = oracle.quant_weight_block(d["W"], 0)
    q, s = fq.quant_weight_block(dev_bf16(d["W"]), "f32")
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), sw)
    out = fq.gemm_w8a8_block(dev_u8(aq), dev_f32(sa), dev_u8(wq), dev_f32(sw), 0)
    assert fq.check_device_error() == 0
    ref, absref = oracle.gemm_w8a8_block(aq, sa, wq, sw, 0)
    assert_within_gemm_tolerance(host_bf16_f64(out), ref, absref, "after timeout",
                                 steps=promoted_steps(aq.shape[1]))


def test_repeated_timeouts():
    for _ in range(3):
        fq.selftest_timeout(500_000)
        assert fq.check_device_error() == fq.FP8Q_ERR_TIMEOUT


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 16), (128, 7), (64, 1)])
def test_tree_attention_whose_waits_run_out(D, bs):
    """The tree attention itself with waits of a few polls (4 us each).  NaN values of drafted nodes keep
    the softmax warps busy for longer than that, so that waits of the other roles run out with copies
    and products in flight.  The status is FP8Q_ERR_TIMEOUT, or the call got through and its results are
    the ordinary call's; the next ordinary call is right either way, and rows behind the last sequence
    stay as they were."""
    Hq, Hkv, rng = 8, 2, np.random.default_rng(5)
    n, ctx, most = np.array([700, 0, 1, 90, 400]), np.array([300, 70, 2500, 1111, 0]), 2540
    need = -(-(ctx + n) // bs)
    perm = rng.permutation(int(need.sum()))
    table = np.zeros((len(n), -(-most // bs)), np.int32)
    at = 0
    for b in range(len(n)):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    codes = lambda *shape: rng.integers(0x20, 0x50, shape).astype(np.uint8)
    total = int(n.sum())
    v = codes(at * bs, Hkv * D)
    for p in range(ctx[0], ctx[0] + n[0], 50):
        v[table[0, p // bs] * bs + p % bs, p % (Hkv * D)] = 0x7F
    args = (dev_u8(codes(total + 3, Hq * D)), dev_u8(codes(at * bs, Hkv * D)), dev_u8(v),
            dev_f32(np.array([0.01, 0.01, 0.01], np.float32)), i32(table), i32(ctx),
            i32(np.concatenate([[0], np.cumsum(n)])), None, Hq, Hkv, bs, 700, most)
    out = torch.full((total + 3, Hq * D), 3.0, dtype=torch.bfloat16, device="cuda")
    bits = lambda t: t.view(torch.int16)                         # NaN among them
    want = fq.attention_tree(*args, out=out.clone())
    assert fq.check_device_error() == 0 and want.isnan().any() and not want.isnan().all()
    seen = []
    for polls in (1, 1, 1, 2, 3, 4, 6, 9, 14, 1 << 18):
        got = fq.selftest_attention_tree(polls, *args, out=out.clone())
        seen.append(fq.check_device_error())
        assert seen[-1] in (0, fq.FP8Q_ERR_TIMEOUT)
        if seen[-1] == 0:
            assert torch.equal(bits(got), bits(want))
        assert (got[total:] == 3.0).all()
        again = fq.attention_tree(*args, out=out.clone())
        assert fq.check_device_error() == 0 and torch.equal(bits(again), bits(want))
    assert seen[:3] == [fq.FP8Q_ERR_TIMEOUT] * 3 and seen[-1] == 0
