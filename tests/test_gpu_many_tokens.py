"""Sizes past what one launch takes: a grid of 2^32 threads or more wraps without
an error. Rows repeat a block of 1024, so that the whole output can be checked
against that block's."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routing_grouped_gemm_router_amd as moe

N = 1024
T = (1 << 26) + N + 5                       # a wave a token: 2^32 threads and more


def _block(shape, seed, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if dtype is torch.uint8:
        return torch.randint(0, 256, shape, generator=g, dtype=dtype, device="cuda")
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _over(block):
    return block.repeat((T + N - 1) // N, 1)[:T]


def _same(big, block):
    """Whether every row of big is its row of the repeated block."""
    whole = big.shape[0] // N * N
    ok = torch.equal(big[whole:], block[:big.shape[0] - whole])
    return ok and all((p == block).all() for p in big[:whole].view(-1, *block.shape).split(4096))


def _mirrored():
    """token_pos of T tokens, each to the mirror of its row."""
    return torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")[:, None]


@pytest.mark.parametrize("mx", [False, True])
def test_permute(mx):
    x = _block((N, 32), 1, torch.uint8 if mx else torch.bfloat16)
    pos = _mirrored()
    if mx:
        s = _block((N, 1), 2, torch.uint8)
        got, gs = moe.moe_permute(_over(x), pos, x_scale=_over(s))
        assert _same(gs.flip(0), s)
    else:
        got = moe.moe_permute(_over(x), pos)
    assert _same(got.flip(0), x)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_combine(dt):
    y, gate = _block((N, 32), 3, dt), _block((N, 1), 4, torch.float32)
    out = moe.moe_combine(_over(y).flip(0), _over(gate), _mirrored())
    assert _same(out, (y.float() * gate).to(dt))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [4096, 4096 - 32])
def test_quantise_rows(dt, cols):
    """2^36 elements, gathered from the block's rows: two threads a block of 32."""
    rows = (1 << 36) // cols + N + 5
    torch.cuda.empty_cache()
    x = _block((N, cols), 5, dt)
    q, s = moe.mxfp8_quantize(x, 1)
    got, gs = moe.mxfp8_quantize(x, 1, row_map=torch.arange(rows, dtype=torch.int32, device="cuda") % N)
    assert _same(got, q) and _same(gs, s)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_quantise_whole_rows(dt):
    """The rows' own order over several launches: 2^33 elements each."""
    rows, cols = (1 << 22) + N + 5, 4096
    torch.cuda.empty_cache()
    x = _block((N, cols), 7, dt)
    big = torch.empty(rows, cols, dtype=dt, device="cuda")
    big[:rows // N * N].view(-1, N, cols).copy_(x.expand(rows // N, N, cols))
    big[rows // N * N:] = x[:rows % N]
    got, gs = moe.mxfp8_quantize(big, 1)
    q, s = moe.mxfp8_quantize(x, 1)
    assert _same(got, q) and _same(gs, s)


def test_route():
    """2^29 tokens of two experts, eight threads a token: every token's row is its
    own, the rows of an expert in the order of their tokens."""
    M, rep = 1 << 20, (1 << 9) + 1
    torch.cuda.empty_cache()
    block = _block((M, 2), 6, torch.float32)
    tokens = M * rep
    r = moe.moe_route(block.repeat(rep, 1), 1)
    idx = (block[:, 1] > block[:, 0]).int()
    ones = int(idx.sum())
    assert r["counts"].tolist() == [rep * (M - ones), rep * ones] and r["offsets"].tolist() == [0, rep * (M - ones), tokens]
    # a token's row: those of its expert in its block before it, and in the blocks before that
    rank = torch.where(idx == 1, idx.cumsum(0), (1 - idx).cumsum(0)) - 1
    first = torch.where(idx == 1, rep * (M - ones), 0) + rank
    step = torch.where(idx == 1, ones, M - ones)
    for i in (0, 1, 2, rep // 2, rep - 2, rep - 1):
        at = slice(i * M, (i + 1) * M)
        pos = r["token_pos"][at, 0]
        assert torch.equal(pos.long(), first + i * step)
        assert torch.equal(r["topk_idx"][at, 0], idx) and (r["topk_gate"][at] == 1).all()
        assert torch.equal(r["sorted_token"][pos.long()], torch.arange(i * M, (i + 1) * M, dtype=torch.int32, device="cuda"))


def test_load_balance():
    """2^30 tokens of two experts, four threads a token. With the block's counts times
    the repetitions f (3/4 and 1/4) and P stay as they are: P's sums are fp32 in a chunk
    of 64 tokens, the same on both sides, and fp64 from there on, and a statistic is
    rounded once. The gradient is the block's divided by the repetitions: its factor
    alpha E / T and two products round here and the comparison's product does, one
    product rounds there (its factor is a power of two): 5 u."""
    M, rep, u = 1 << 20, (1 << 10) + 1, 2.0 ** -24
    torch.cuda.empty_cache()
    block = _block((M, 2), 8, torch.float32)
    counts = torch.tensor([3 << 18, 1 << 18], dtype=torch.int32, device="cuda")
    d1 = torch.zeros_like(block)
    want = moe.moe_load_balance(block, counts, 1, 0.5, dlogits=d1)
    big = block.repeat(rep, 1)
    d = torch.zeros_like(big)
    got = moe.moe_load_balance(big, counts * rep, 1, 0.5, dlogits=d)
    assert torch.allclose(got, want, rtol=2 * u, atol=0)
    for part in d.view(rep, M, 2).split(64):
        assert ((part * rep - d1).abs() <= 5 * u * d1.abs() + 1e-35).all()
