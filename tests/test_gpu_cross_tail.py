"""Cross attention of long sequences whose states weigh next to nothing one by one and something
together."""
import numpy as np
import pytest
import torch

from paged_kv_cache_231_gb300 import binding as B

from .step_util import DEV, half_step, i32

pytestmark = pytest.mark.gpu
N, BS, HKV = 60000, 16, 8


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("d,g,batch,rows", [(128, 4, 160, 1), (64, 1, 160, 1), (128, 1, 40, 200),
                                            (64, 2, 40, 40)])
def test_many_states_of_little_weight(d, g, batch, rows, dtype):
    # One state of score 0 and value 0, N - 1 of score -s and values around 1, the same for every
    # sequence (they share the blocks), and many sequences, so that one unit goes through most of
    # a sequence. Weights: 1 and e^-s = 2^-25.1 to 2^-24.4; out = sum of w v / (1 + sum of w).
    gen = torch.Generator()
    gen.manual_seed(d + rows)
    blocks = N // BS
    k = torch.zeros((blocks, BS, HKV, d))
    k[..., 0] = -torch.empty((blocks, BS, HKV)).uniform_(16.9, 17.4, generator=gen)
    v = torch.empty((blocks, BS, HKV, d)).uniform_(0.5, 1.5, generator=gen)
    k[0, 0], v[0, 0] = 0.0, 0.0
    k, v = k.to(dtype), v.to(dtype)
    q = torch.zeros((batch * rows, HKV * g, d), dtype=dtype)
    q[..., 0] = 1.0
    lse = torch.empty((batch * rows, HKV * g), device=DEV)
    table = i32(np.tile(np.arange(blocks, dtype=np.int32), (batch, 1)))
    out = B.pkv_cross_attention(
        q.view(batch * rows, -1).to(DEV), k.to(DEV), v.to(DEV), i32(np.arange(batch + 1) * rows),
        i32([N] * batch), table, num_heads=HKV * g, kv_num_heads=HKV, max_query_len=rows,
        scale=1.0, lse=lse)
    torch.cuda.synchronize()
    w = torch.exp(k[..., 0].double()).view(N, HKV)
    total = w.sum(0)
    ref = torch.einsum("nh,nhd->hd", w, v.double().view(N, HKV, d)) / total[:, None]
    got = out.cpu().double().view(batch * rows, HKV, g, d)
    # A weight: scores of one product, exact in fp32, scaled by log2 e (below 26, half steps of
    # 2^-20 relative to the weight), exp2 to 2^-21, one rounding to dtype; in fp16 at least 2^-25
    # against a largest weight of 2^7 or more, so 2^-32 * N of the whole. N terms in fp32: the
    # partial sums of a step are formed by the tensor core, each addition errs by 2^-23 of the sum
    # (twice half a step, for cut digits): N * 2^-23. The result is rounded once.
    half = half_step(dtype)
    size = ref.abs()
    tol = size * (half * 2.02 + 2.0 ** -19 + (N + 64) * 2.0 ** -23)
    if dtype is torch.float16:
        tol = tol + N * 2.0 ** -32 * 1.5
    err = (got - ref[None, :, None]).abs()
    assert (err <= tol[None, :, None]).all(), (float(err.max()), float(tol.min()))
    want = torch.log(total)[None, :, None].expand(-1, -1, g).reshape(1, -1)
    assert ((lse.cpu().double() - want).abs() <= (N + 64) * 2.0 ** -23 + 2.0 ** -19).all()
