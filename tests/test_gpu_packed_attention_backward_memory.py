"""dflash_packed_block_attention_backward's shares of the context gradients: how
much memory they take, and fp32 sums that are moved to memory on the way.

Tolerances: the tensor cores truncate by at most 2^-23 of a sum a step, 2^-24 on
average, and 96 steps follow one another before a sum starts again; e^ and lse
add 2^-20 of independent terms."""
import math

import pytest
import torch

from test_packed_attention_backward_cpu import backward_reference, forward_reference, operands

pytestmark = pytest.mark.gpu


def _df():
    import block_diffusion_drafter_dflash_gb300 as df
    return df


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,g,S,nq,nkv", [(512, 16, 4096, 32, 8), (4096, 16, 32768, 32, 8), (8191, 16, 65536, 32, 8),
                                          (8191, 32, 1000, 8, 1), (3, 4, 100, 4, 2)])
def test_workspace_follows_the_operands(N, g, S, nq, nkv, hd, dtype):
    """Laid-out operands (two or four bytes a value), three statistics a query row, and fp32 shares of both context
    gradients: at most eight items an SM and one for each kv head and key tile, 128 rows each."""
    from block_diffusion_drafter_dflash_gb300 import _abi
    size = int(_df().lib().dflash_packed_attention_backward_workspace_bytes(
        N, g, S, nq, nkv, hd, _abi.DTYPE_F32 if dtype == torch.float32 else _abi.DTYPE_BF16))
    rows, ctx = -(-N // (128 // g)) * 128, -(-S // 128) * 128
    value = 4 if dtype == torch.float32 else 2
    operand = value * hd * (2 * rows * nq + 2 * ctx * nkv + 2 * rows * nkv)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    shares = 2 * 4 * hd * 128 * (8 * sms + 2 * nkv * (ctx // 128))
    assert 0 < size <= operand + 12 * rows * nq + shares + 8 * N + 4 * rows + (1 << 16)


# blocks of 16 unless said; context items of 10, 16, 24 and 63 streamed tiles on 152 SMs, sums moved to memory every 8
# (heads of 128) or 12 (64): in the middle, at the end, and seven times
CASES = [(130, 400, 16, 8, 1, 128), (200, 608, 16, 8, 1, 128), (1000, 456, 16, 8, 1, 64), (1500, 400, 16, 8, 2, 128),
         (1500, 401, 9, 8, 2, 64)]


@pytest.mark.parametrize("S,N,g,nq,nkv,hd", CASES)
def test_fp32_sums_moved_to_memory(S, N, g, nq, nkv, hd):
    df = _df()
    for anchors in ([S] * N, torch.randint(0, S + 1, (N,), generator=torch.Generator().manual_seed(3)).tolist()):
        ops = operands(S, N, g, nq, nkv, hd, torch.float32, 14, "cuda")
        d_out = torch.randn(ops[0].shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
        ref = [t.double() for t in ops]
        out, lse, _ = forward_reference(*ref, anchors)
        out, lse = out.float().contiguous(), lse.float().contiguous()
        a = torch.tensor(anchors, dtype=torch.int32, device="cuda")
        ws = df.dflash_packed_attention_backward_workspace(N, g, S, nq, nkv, hd, torch.float32)
        twice = []
        for _ in range(2):
            ws.fill_(255)                                  # NaN wherever a value is read before it is written
            grads = [torch.full_like(t, math.nan) for t in ops]
            df.dflash_packed_block_attention_backward(*ops, a, out, lse, d_out, *grads, ws)
            assert df.dflash_packed_attention_status(ws) == 0
            twice.append(grads)
        assert all(torch.equal(x, y) for x, y in zip(*twice))
        for name, got, w in zip(("d_q", "d_k_ctx", "d_v_ctx", "d_k_blk", "d_v_blk"), twice[0],
                                backward_reference(*ref, anchors, d_out.double())):
            err = float((got.double() - w).norm() / w.norm())
            print(f"{name}: rel {err:.2e}")
            assert err <= 96 * 2.0 ** -24 + 2.0 ** -20, name
