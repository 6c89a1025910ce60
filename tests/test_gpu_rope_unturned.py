"""Dims beside the rotated part of idx_rope: every bit pattern passes unchanged."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scoring_top_amd as idx  # noqa: E402


def bits(n, heads, dtype):
    """Rows [n, heads, 128] of every bit pattern: NaN, infinities and subnormals among them."""
    count = n * heads * 128
    if dtype is torch.bfloat16:
        x = torch.arange(count, dtype=torch.int32).to(torch.int16)
    else:
        rng = np.random.default_rng(1)
        x = rng.integers(0, 1 << 32, count, dtype=np.uint64).astype(np.uint32)
        x[::5] |= 0x7F800000          # infinities and NaN of both kinds
        x[::7] &= 0x807FFFFF          # zeros and subnormals
        x = torch.from_numpy(x.view(np.int32))
    return x.view(n, heads, 128).view(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("rot,first", [(64, 0), (64, 64), (16, 56), (112, 8)])
def test_unturned_dims_keep_their_bits(rot, first, adjacent, dtype):
    n = 64
    q, k = bits(n, 8, dtype), bits(n, 2, dtype)
    q[..., first:first + rot] = 1
    k[..., first:first + rot] = 1
    tok_len = torch.arange(1, n + 1, dtype=torch.int32, device="cuda")
    out = idx.idx_rope(q.cuda(), k.cuda(), tok_len, idx.idx_rope_table(rot), first=first,
                       interleaved=adjacent)
    rest = [d for d in range(128) if not first <= d < first + rot]
    word = torch.int16 if dtype is torch.bfloat16 else torch.int32
    for got, x in zip(out, (q, k)):
        assert torch.equal(got.cpu().view(word)[..., rest], x.view(word)[..., rest])
