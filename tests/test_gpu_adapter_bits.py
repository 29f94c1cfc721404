"""All 24 bits of the adapters' fp32 h and dh through the products that take them in three bf16 parts.

Every value compared is one product of powers of two with one h or dh, so it is exact in fp32 whatever the order of sums; and every h and dh is an
odd number of 23 or 24 bits (an odd 8-bit weight times an odd 16-bit scale), so that its third part is not zero and is its own: a part that is
missing, of another rank or of another row shows in the bits.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    yield split_gemm_gb300
    assert split_gemm_gb300.adapter_status() == 0


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def sign(self, *shape):
        return 2.0 * torch.randint(0, 2, shape, generator=self.g) - 1

    def odd(self, lo, hi, *shape):
        return (2 * torch.randint(lo // 2, hi // 2, shape, generator=self.g) + 1).float() * self.sign(*shape)

    def power(self, *shape):
        return 2.0 ** torch.randint(0, 3, shape, generator=self.g) * self.sign(*shape)

    def index(self, rows, adapters):
        """Rows anywhere, some adapters with many of them; some rows have none."""
        e = (adapters * torch.rand(rows, generator=self.g) ** 2).long().clamp(max=adapters - 1)
        return torch.where(torch.rand(rows, generator=self.g) < 0.1, -1, e)

    def one_hot(self, rows, cols):
        return torch.zeros(rows, cols).scatter_(1, torch.randint(cols, (rows, 1), generator=self.g), self.power(rows, 1))

    def one_of_each(self, lines, rank):
        """[lines, rank], a power of two in one place of each line, every place taken where the lines do."""
        at = torch.arange(lines) % rank
        return torch.zeros(lines, rank).scatter_(1, at[torch.randperm(lines, generator=self.g)].unsqueeze(1), self.power(lines, 1))

    def one_row_to_a_column(self, index, adapters, cols):
        """[rows, cols], in each column a power of two in one row of each adapter that has rows."""
        v = torch.zeros(len(index), cols)
        for e in range(adapters):
            mine = (index == e).nonzero()[:, 0]
            if len(mine):
                v[mine[torch.randint(len(mine), (cols,), generator=self.g)], torch.arange(cols)] = self.power(cols)
        return v


def _by_adapter(u, weights, index):
    """u[t] @ weights[e] in 64 bits for each row t of an adapter e, zeros for the others."""
    out = torch.zeros(len(index), weights.shape[2], dtype=torch.float64)
    for e, w in enumerate(weights.double()):
        out[index == e] = u[index == e].double() @ w
    return out


def _sums(u, v, index, adapters):
    """[adapters, ...]: the sum of u[t] v[t]^T over each adapter's rows."""
    return torch.stack([u[index == e].double().T @ v[index == e].double() for e in range(adapters)])


def _third_part(v):
    """The bits of a value's 24 that its first 16 do not hold, of what is not zero."""
    m, _ = np.frexp(v[v != 0])
    return np.ldexp(np.abs(m), 24).astype(np.int64) & 0xff


def _same(got, want):
    want = want.numpy()
    assert np.array_equal(got.cpu().double().numpy(), want), f"{np.count_nonzero(got.cpu().double().numpy() != want)} of {want.size} differ"


def _grads(sg, rows, cols, outs, rank, adapters, x_type):
    """dx and da, with what they have to be."""
    d = Draw(rows + 3 * cols + 5 * outs + 7 * rank)
    index = d.index(rows, adapters)
    b, dy = d.odd(129, 255, adapters, outs, rank), d.one_hot(rows, outs)
    a = torch.stack([d.one_of_each(cols, rank).T for _ in range(adapters)])
    scale = d.odd(32769, 65535, adapters) / 65536
    x = d.one_row_to_a_column(index, adapters, cols)
    dh = _by_adapter(dy, b.double() * scale.double()[:, None, None], index)
    assert (dh[index >= 0] != 0).all() and _third_part(dh.numpy()).all()
    plan = sg.adapter_plan(index.int().cuda(), adapters)
    xd = x.to(BF16).cuda()
    got = sg.adapter_bwd(dy.to(BF16).cuda(), sg.mxint8_quantize(xd) if x_type == "int8" else xd, torch.zeros(rows, rank, device="cuda"),
                         a.to(BF16).contiguous().cuda(), b.to(BF16).cuda(), plan, scale.cuda(), out_dtype=F32)
    return got[:2], (_by_adapter(dh, a, index), _sums(dh, x, index, adapters))


# rows, cols, outs, rank, adapters; ranks that are no multiple of 4, whose dh the sums read by single elements while the pass that makes it has only just ended
@pytest.mark.parametrize("shape", [(50, 64, 40, 1, 2), (700, 96, 72, 5, 3), (900, 264, 33, 7, 2), (1300, 200, 136, 33, 4), (2500, 72, 64, 78, 2), (600, 333, 101, 127, 3)])
@pytest.mark.parametrize("x_type", ["bf16", "int8"])
def test_dh_of_ranks_that_are_not_whole_vectors(sg, shape, x_type):
    for _ in range(3):
        for got, want in zip(*_grads(sg, *shape, x_type)):
            _same(got, want)


# One token to many tiles, each way that rows are cut up: few rows (rank up to 64), tiles of 64 and of 128 rows, clusters of 1 to 8; whole vectors
# and not; 8 to 128 ranks, odd numbers of sixteens and eights among them; one stage of a sum and many, odd numbers and even
SHAPES = [(1, 64, 136, 16, 1), (9, 1001, 72, 33, 2), (40, 200, 96, 24, 3), (300, 96, 264, 16, 4), (160, 72, 200, 64, 3),
          (700, 256, 520, 32, 3), (641, 101, 333, 17, 3), (161, 72, 200, 64, 1), (129, 136, 264, 100, 3), (5, 4096, 512, 128, 2), (130, 64, 392, 128, 2),
          (1500, 136, 200, 72, 2), (1300, 1001, 136, 20, 2), (2049, 64, 136, 64, 1), (3000, 384, 384, 48, 2), (2500, 72, 333, 90, 5), (12544, 64, 128, 16, 1)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("scaled", [True, False])
def test_forward(sg, shape, scaled):
    """out = b h where h has 24 bits: an odd weight times an odd scale, or two of x's columns whose products lie 2^15 apart."""
    rows, cols, outs, rank, adapters = shape
    d = Draw(rows + 3 * cols + 5 * outs + 7 * rank)
    index = d.index(rows, adapters) if rows > 1 else torch.zeros(1, dtype=torch.long)
    a = d.odd(129, 255, adapters, rank, cols)
    b = torch.stack([d.one_of_each(outs, rank) for _ in range(adapters)])
    x, scale = d.one_hot(rows, cols), None
    if scaled:
        scale = d.odd(32769, 65535, adapters) / 65536
    else:  # the second column of a row: some other one, its value 2^-15 of the first's
        at = x.abs().argmax(1, keepdim=True)
        x = x.scatter(1, (at + 1 + torch.randint(cols - 1, (rows, 1), generator=d.g)) % cols, x.gather(1, at) * 2.0 ** -15)
    h = _by_adapter(x, a.transpose(1, 2).double() * (1.0 if scale is None else scale.double()[:, None, None]), index)
    assert (h.float().double() == h).all() and (_third_part(h.numpy()) != 0).mean() > 0.9
    plan = sg.adapter_plan(index.int().cuda(), adapters)
    out, got_h = sg.adapter_fwd(torch.zeros(rows, outs).cuda(), x.to(BF16).cuda(), a.to(BF16).cuda(), b.to(BF16).cuda(), plan,
                                None if scale is None else scale.cuda())
    _same(got_h, h)
    _same(out, _by_adapter(h, b.transpose(1, 2), index))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("x_type", ["bf16", "int8"])
def test_dx_and_da(sg, shape, x_type):
    for got, want in zip(*_grads(sg, *shape, x_type)):
        _same(got, want)


@pytest.mark.parametrize("shape", SHAPES)
def test_db(sg, shape):
    """h of 24 bits that no other row, rank or part of one has; dy with one row of each adapter to a column."""
    rows, cols, outs, rank, adapters = shape
    d = Draw(rows + 3 * cols + 5 * outs + 7 * rank)
    index = d.index(rows, adapters)
    h, dy = d.odd(2 ** 23, 2 ** 24 - 1, rows, rank), d.one_row_to_a_column(index, adapters, outs)
    assert (_third_part(h.numpy()) != 0).all()
    zeros = torch.zeros(adapters, rank, cols, dtype=BF16).cuda(), torch.zeros(adapters, outs, rank, dtype=BF16).cuda()
    db = sg.adapter_bwd(dy.to(BF16).cuda(), torch.zeros(rows, cols, dtype=BF16).cuda(), h.cuda(), *zeros,
                        sg.adapter_plan(index.int().cuda(), adapters))[2]
    _same(db, _sums(dy, h, index, adapters))
