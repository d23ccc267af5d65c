"""qs_apply_adapters (through the binding) against the oracle in fp64.

Tolerances, with u = 2^-24 (half a float32 step): products of two bf16 values are exact
in float32. A coordinate (down x) is a sum of K of them, split over lanes, at most
K / 16 + 16 additions to a lane and the joins: u (K / 16 + 16) sum|down x|; the scale
one rounding more. It enters the product with `up` as three bf16 numbers whose sum it
is, so that there are at most 3 rank additions and the logit's own, and the result is
rounded once to float32 and once to its type (half a step: u, bf16 2^-8).
"""

import numpy as np
import pytest

import oracle
from test_gpu_score import bf16, on_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def qs():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_sampling_vocabs_amd as qs
    qs.load()
    return qs


def half(x):
    """Exactly representable bf16 values, and their float64."""
    return bf16(np.asarray(x, np.float32))


def inputs(seed, B, V, K, rank, count):
    rng = np.random.default_rng(seed)
    z = bf16(rng.normal(0, 3, (B, V)))
    x = half(rng.normal(0, 1, (B, K)))
    down = half(rng.normal(0, K ** -0.5, (count, rank, K)))
    up = half(rng.normal(0, rank ** -0.5, (count, V, rank)))
    scale = rng.uniform(0.5, 2.0, count).astype(np.float32)
    index = rng.integers(-1, count, B).astype(np.int32)
    return z, x, down, up, scale, index


def to(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def to16(x):
    import torch
    return to(x).to(torch.bfloat16)


def check(z, dtype, x, down, up, scale, index, got):
    B = z.shape[0]
    K, rank = x.shape[1], down.shape[1]
    g = got.float().cpu().numpy().astype(np.float64)
    step = U if dtype == "f32" else 2.0 ** -8
    for b in range(B):
        a = int(index[b])
        if a < 0 or a >= down.shape[0]:
            assert np.array_equal(g[b], z[b].astype(np.float64)), b
            continue
        s = 1.0 if scale is None else float(scale[a])
        want = oracle.adapted_row(z[b], x[b], down[a], up[a], s)
        d, w = np.abs(down[a].astype(np.float64)), np.abs(up[a].astype(np.float64))
        u = down[a].astype(np.float64) @ x[b].astype(np.float64)
        e_u = abs(s) * U * (K / 16 + 18) * (d @ np.abs(x[b].astype(np.float64)))
        size = np.abs(z[b].astype(np.float64)) + w @ (abs(s) * np.abs(u))
        tol = w @ e_u + U * (3 * rank + 6) * size + (U + step) * np.abs(want)
        bad = ~(np.abs(g[b] - want) <= 1.01 * tol)
        assert not bad.any(), (b, np.nonzero(bad)[0][:4], g[b][bad][:4], want[bad][:4], tol[bad][:4])


def run(qs, z, dtype, x, down, up, scale, index, in_place=True, extra=1, **kw):
    import torch
    lg = on_gpu(z, dtype, extra)
    out = None if in_place else on_gpu(np.zeros_like(z), dtype, extra)
    status = qs.apply_adapters(lg, to16(x), to16(down), to16(up), to(index),
                               None if scale is None else to(scale), out=out, **kw)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(lg.float().cpu(), torch.from_numpy(z)), "the input has changed"
    return (lg if in_place else out), status


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 3, 15, 16, 17, 63, 64, 65, 127, 255, 257, 1000, 4099, 32003])
def test_sizes(qs, V, dtype, in_place):
    for B, K, rank, count in ((1, 64, 8, 1), (5, 136, 16, 3), (17, 512, 40, 4), (64, 256, 64, 9)):
        print(f"adapters V={V} {dtype} B={B} K={K} rank={rank}", flush=True)
        case = inputs(V + B, B, V, K, rank, count)
        got, status = run(qs, case[0], dtype, *case[1:], in_place=in_place)
        assert not status.any()
        check(case[0], dtype, *case[1:], got)


@pytest.mark.parametrize("rank", list(range(8, 129, 8)))
def test_ranks(qs, rank):
    for dtype in ("f32", "bf16"):
        print(f"adapters rank={rank} {dtype}", flush=True)
        case = inputs(rank, 19, 777, 200, rank, 5)
        got, _ = run(qs, case[0], dtype, *case[1:], in_place=False)
        check(case[0], dtype, *case[1:], got)


@pytest.mark.parametrize("K", [8, 16, 24, 120, 512, 520, 2048, 4104, 8192, 65536])
def test_widths(qs, K):
    print(f"adapters K={K}", flush=True)
    case = inputs(K, 3, 300, K, 16, 3)
    got, _ = run(qs, case[0], "f32", *case[1:])
    check(case[0], "f32", *case[1:], got)


@pytest.mark.parametrize("B", [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 128, 200])
@pytest.mark.parametrize("kind", ["own", "one", "none", "mixed"])
def test_batches(qs, B, kind):
    """Every row its own adapter, all the same, none at all, and any."""
    print(f"adapters B={B} {kind}", flush=True)
    z, x, down, up, scale, index = inputs(B, B, 501, 128, 8, max(B, 2))
    index = {"own": np.random.default_rng(B).permutation(B), "one": np.full(B, 1),
             "none": np.full(B, -1), "mixed": index}[kind].astype(np.int32)
    for in_place in (True, False):
        got, status = run(qs, z, "bf16", x, down, up, scale, index, in_place=in_place)
        assert not status.any()
        check(z, "bf16", x, down, up, scale, index, got)
    again, _ = run(qs, z, "bf16", x, down, up, None, index)
    check(z, "bf16", x, down, up, None, index, again)


@pytest.mark.parametrize("B,count", [(65, 1), (320, 64), (700, 5), (4096, 300), (4161, 3),
                                     (9000, 70)])
def test_more_rows_than_a_block(qs, B, count):
    """Batches whose rows are put in order over blocks of 64 (and over 4096 rows, one order
    behind another), with rows without an adapter and bad indexes among them."""
    print(f"adapters B={B} count={count}", flush=True)
    z, x, down, up, scale, index = inputs(B, B, 70, 32, 16, count)
    index[::17] = count + 3
    index[5::23] = -5
    bad = (index < -1) | (index >= count)
    for in_place in (True, False):
        got, status = run(qs, z, "bf16", x, down, up, scale, index, in_place=in_place)
        assert np.array_equal(status.cpu().numpy(), np.where(bad, 4, 0))
        check(z, "bf16", x, down, up, scale, index, got)


def test_bad_indexes(qs):
    """An index that is no adapter leaves the row as it is and is reported."""
    z, x, down, up, scale, index = inputs(1, 9, 300, 64, 16, 4)
    index[:] = [0, 4, -2, 3, np.iinfo(np.int32).max, np.iinfo(np.int32).min, -1, 2, 5]
    for in_place in (True, False):
        got, status = run(qs, z, "f32", x, down, up, scale, index, in_place=in_place)
        assert status.tolist() == [0, 4, 4, 0, 4, 4, 0, 0, 4]
        check(z, "f32", x, down, up, scale, index, got)
    # no adapters at all
    index[:] = -1
    index[3] = 0
    got, status = run(qs, z, "f32", x, down[:0], up[:0], scale[:0], index)
    assert status.tolist() == [0, 0, 0, 4, 0, 0, 0, 0, 0]
    assert np.array_equal(got.cpu().numpy(), z)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_padding(qs, dtype):
    """Factors and hidden states inside larger tensors, adapters in any order, and what
    lies behind a row's last logit."""
    import torch
    B, V, K, rank, count = 18, 333, 96, 24, 5
    z, x, down, up, scale, index = inputs(3, B, V, K, rank, count)
    big_d = torch.full((count, rank + 3, K + 16), 9.0, dtype=torch.bfloat16, device="cuda")
    big_u = torch.full((count * 2, V + 5, rank + 40), 9.0, dtype=torch.bfloat16, device="cuda")
    big_x = torch.full((B + 2, K + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    d, u, h = big_d[:, :rank, :K], big_u[::2, 2:V + 2, 8:rank + 8], big_x[1:B + 1, :K]
    d.copy_(to16(down))
    u.copy_(to16(up))
    h.copy_(to16(x))
    lg = on_gpu(z, dtype, extra=2)
    base = lg._base if lg._base is not None else lg
    behind = base[:, V:].clone()
    status = qs.apply_adapters(lg, h, d, u, to(index), to(scale))
    torch.cuda.synchronize()
    assert not status.any()
    check(z, dtype, x, down, up, scale, index, lg)
    assert torch.equal(base[:, V:], behind)
    # one adapter for every row through a stride of 0, and views of single elements
    one = qs.apply_adapters(on_gpu(z, dtype), h, d[1:2].expand(4, -1, -1),
                            u[1:2].expand(4, -1, -1), to(np.full(B, 3, np.int32)))
    assert not one.any()
    lg = on_gpu(z[:1], dtype)
    qs.apply_adapters(lg, h[:1], d[2:3], u[2:3], to(np.zeros(1, np.int32)))
    check(z[:1], dtype, x[:1], down[2:3], up[2:3], None, np.zeros(1, np.int32), lg)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_do_not_meet(qs, dtype):
    """Infinities and NaN in one adapter, hidden state or logit stay with their rows, and
    with their logits where they are the up factor's."""
    B, V, K, rank, count = 40, 700, 128, 16, 6
    z, x, down, up, scale, index = inputs(5, B, V, K, rank, count)
    index = (np.arange(B) % 6).astype(np.int32)
    index[7] = -1
    z[7, :3] = [np.nan, np.inf, -np.inf]
    z[8, 5] = np.inf
    want, _ = run(qs, z, dtype, x, down, up, scale, index)
    want = want.float().cpu().numpy()
    up[3, 11, 2] = np.inf
    down[4, 0, 0] = np.nan
    scale[5] = np.inf
    x[0, 1] = np.inf
    got, _ = run(qs, z, dtype, x, down, up, scale, index)
    got = got.float().cpu().numpy()
    for b in range(B):
        a = index[b]
        if a in (4, 5) or b == 0:
            assert not np.isfinite(got[b]).any(), b
        elif a == 3:
            assert not np.isfinite(got[b, 11]), b
            keep = np.arange(V) != 11
            assert np.array_equal(got[b, keep], want[b, keep], equal_nan=True), b
        else:
            assert np.array_equal(got[b], want[b], equal_nan=True), b


@pytest.mark.parametrize("rank", [8, 16, 24, 40, 128])
def test_infinite_coordinates(qs, rank):
    """An infinite coordinate times the factors is what the formula says: infinities, and
    NaN where they cancel or meet a 0."""
    B, V, K, count = 3, 70, 64, 2
    z, x, down, up, scale, index = inputs(rank, B, V, K, rank, count)
    index[:] = [0, 1, -1]
    x[0, 5] = np.inf          # with factors of either sign
    scale[1] = np.inf
    up[:, :30] = np.abs(up[:, :30])
    up[:, 30:60] = -np.abs(up[:, 30:60])
    up[0, 3, rank // 2] = 0
    down[0, :, 5] = 0.5
    down[1] = np.abs(down[1])
    x[1] = np.abs(x[1])
    got, status = run(qs, z, "f32", x, down, up, scale, index)
    assert (status.cpu() == 0).all()
    got = got.cpu().numpy()
    for b in (0, 1):
        assert (got[b, 30:60] == -np.inf).all(), b
        assert (np.delete(got[b, :30], 3) == np.inf).all(), b
        with np.errstate(invalid="ignore"):
            mixed = up[b, 60:].astype(np.float64) @ np.full(rank, np.inf)
        assert np.array_equal(got[b, 60:].astype(np.float64), mixed, equal_nan=True), b
    assert np.isnan(got[0, 3]) and got[1, 3] == np.inf
    assert np.array_equal(got[2], z[2])


@pytest.mark.parametrize("rank", [8, 16, 32, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_largest_coordinates(qs, rank, sign):
    """Coordinates past the largest bf16 number: 2^127 (1 + 255/256 + 1/512)."""
    B, V, K, count = 2, 40, 16, 1
    z, x, down, up, scale, index = inputs(9, B, V, K, rank, count)
    x[:], down[:] = 0, 0
    x[:, 0], x[:, 1] = sign * 2.0 ** 127, sign * 2.0 ** 120
    down[:, :, 0], down[:, :, 1] = 1.9921875, 0.75
    up = half(up * 2.0 ** -126)
    index[:] = 0
    got, _ = run(qs, z, "f32", x, down, up, None, index)
    check(z, "f32", x, down, up, None, index, got)


@pytest.mark.parametrize("rank", [8, 16, 32, 40])
@pytest.mark.parametrize("e", [-110, -117, -125, -134])
def test_smallest_coordinates(qs, rank, e):
    """Coordinates around 2^e, with factors that make them count: three truncated bf16 terms
    leave less than one's least step, 2^-133, of each."""
    B, V, K, count = 3, 40, 16, 1
    z, x, down, up, _, index = inputs(9, B, V, K, rank, count)
    z[:] = 0
    down = half(down * 2.0 ** e)
    up = half(up * 2.0 ** 100)
    index[:] = 0
    got, _ = run(qs, z, "f32", x, down, up, None, index)
    u = x.astype(np.float64) @ down[0].astype(np.float64).T
    w = up[0].astype(np.float64)
    want = u @ w.T
    # sums and roundings as for other coordinates, whose own products may be subnormal:
    # half a step of 2^-149 for each of K
    e_u = U * (K / 16 + 18) * (np.abs(x) @ np.abs(down[0].astype(np.float64)).T) + K * 2.0 ** -150
    tol = (e_u + 2.0 ** -133) @ np.abs(w).T + U * (3 * rank + 8) * (np.abs(u) @ np.abs(w).T)
    assert (np.abs(got.cpu().numpy() - want) <= 1.01 * tol).all()


def test_same_bits(qs):
    """Twice the same call; and a row's bits whatever rows are beside it, how many there
    are, and where it stands among them."""
    import torch
    for rank in (8, 32, 72):
        z, x, down, up, scale, index = inputs(8, 130, 2001, 256, rank, 12)
        a, _ = run(qs, z, "f32", x, down, up, scale, index)
        b, _ = run(qs, z, "f32", x, down, up, scale, index)
        assert torch.equal(a, b)
        for rows in ([5], [77, 3], list(range(20, 40)), list(range(129, 80, -1)),
                     list(range(60, 124))):
            few, _ = run(qs, z[rows], "f32", x[rows], down, up, scale, index[rows])
            assert torch.equal(few, a[rows]), (rank, rows)


@pytest.mark.parametrize("K", [520, 1032, 2056, 4104, 8192])
@pytest.mark.parametrize("B,rank", [(64, 64), (64, 128), (65, 64), (130, 16), (130, 64)])
def test_widths_of_several_ranks_a_wave(qs, B, rank, K):
    """Widths over several requests of a wave, and over several turns of its loop, where a
    wave takes two ranks (64 rows) or four (more)."""
    print(f"adapters B={B} rank={rank} K={K}", flush=True)
    case = inputs(K + B, B, 72, K, rank, 3)
    got, status = run(qs, case[0], "f32", *case[1:])
    assert not status.any()
    check(case[0], "f32", *case[1:], got)


@pytest.mark.parametrize("rank", [8, 64, 128])
@pytest.mark.parametrize("K", [1032, 2056, 4104])
def test_same_bits_of_wide_rows(qs, K, rank):
    """A row's bits with one, two and four ranks a wave, in batches of any size."""
    import torch
    z, x, down, up, scale, index = inputs(K, 150, 333, K, rank, 5)
    a, _ = run(qs, z, "f32", x, down, up, scale, index)
    for rows in ([5], list(range(20, 40)), list(range(60, 124)), list(range(149, 80, -1))):
        few, _ = run(qs, z[rows], "f32", x[rows], down, up, scale, index[rows])
        assert torch.equal(few, a[rows]), (K, rank, rows)


@pytest.mark.parametrize("rank", [8, 40, 128])
def test_large_batches_of_wide_rows(qs, rank):
    """A thousand rows of several thousand columns against the same rows among 50."""
    import torch
    B, V, K, count = 1025, 4001, 4104, 6
    print(f"adapters B={B} K={K} rank={rank}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(rank)

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    z = rand(B, V + 7).bfloat16()[:, :V]
    x, down, up = (t.bfloat16() for t in (rand(B, K), rand(count, rank, K) / K ** 0.5,
                                          rand(count, V, rank) / rank ** 0.5))
    index = torch.randint(-1, count, (B,), device="cuda", generator=gen, dtype=torch.int32)
    out = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device="cuda")
    status = qs.apply_adapters(z, x, down, up, index, out=out)
    assert not status.any()
    for at in range(0, B, 50):
        rows = slice(at, at + 50)
        qs.apply_adapters(z[rows], x[rows], down, up, index[rows].contiguous())
    assert torch.equal(out, z)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V,rank,count", [(1025, 32003, 8, 40), (1025, 32003, 40, 3),
                                            (257, 32003, 72, 7), (65, 128259, 128, 2)])
def test_large_batches_match_small_ones(qs, B, V, rank, count, dtype):
    """Batches so large that a workgroup goes over several tiles of the vocabulary give
    every row the bits that it has among 64 or fewer; rows without an adapter stay."""
    import torch
    print(f"adapters B={B} V={V} rank={rank} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(B + rank)
    kind = torch.float32 if dtype == "f32" else torch.bfloat16

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    width = (V + 7) // 8 * 8
    z = rand(B, width).to(kind)
    x, down, up = (t.bfloat16() for t in (rand(B, 64), rand(count, rank, 64) / 8,
                                          rand(count, V, rank) / rank ** 0.5))
    index = torch.randint(-1, count, (B,), device="cuda", generator=gen, dtype=torch.int32)
    scale = torch.rand(count, device="cuda", generator=gen) + 0.5
    want = z.clone()
    for at in range(0, B, 50):
        rows = slice(at, at + 50)
        qs.apply_adapters(want[rows, :V], x[rows], down, up, index[rows].contiguous(), scale)
    out = torch.full_like(z, 7.0)
    status = qs.apply_adapters(z[:, :V], x, down, up, index, scale, out=out[:, :V])
    assert not status.any()
    assert torch.equal(out[:, :V], want[:, :V])
    assert bool((out[:, V:] == 7.0).all())
    assert torch.equal(out[index < 0][:, :V], z[index < 0][:, :V])
    assert not torch.equal(out[index >= 0][:, :V], z[index >= 0][:, :V])
    kept = z.clone()
    qs.apply_adapters(z[:, :V], x, down, up, index, scale)
    assert torch.equal(z[:, :V], want[:, :V]) and torch.equal(z[:, V:], kept[:, V:])


def test_inference_mode(qs):
    import torch
    with torch.inference_mode():
        z, x, down, up, scale, index = inputs(8, 5, 300, 64, 8, 3)
        got, status = run(qs, z, "bf16", x, down, up, scale, index)
        assert not status.any()
    check(z, "bf16", x, down, up, scale, index, got)


def test_most_rows(qs):
    """The largest batch, 2^18 rows on two adapters, some rows without: a tile of 16
    batch rows at the end of each block of 64, and every row against float64."""
    import torch
    B, V, K, rank = 1 << 18, 24, 16, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(B, V, generator=g, device="cuda")
    x = torch.randn(B, K, generator=g, device="cuda").bfloat16()
    down = torch.randn(2, rank, K, generator=g, device="cuda").bfloat16()
    up = (torch.randn(2, V, rank, generator=g, device="cuda") / 16).bfloat16()
    index = torch.randint(-1, 2, (B,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.empty_like(z)
    status = qs.apply_adapters(z, x, down, up, index, out=out)
    assert not status.any()
    want = z.double()
    size, sums = torch.zeros_like(want), torch.zeros_like(want)
    for a in range(2):
        on = (index == a)[:, None]
        u = x.double() @ down[a].double().t()
        w = up[a].double()
        want = torch.where(on, want + u @ w.t(), want)
        size = torch.where(on, u.abs() @ w.abs().t(), size)
        # the products that a coordinate is a sum of
        sums = torch.where(on, (x.double().abs() @ down[a].double().abs().t()) @ w.abs().t(), sums)
    tol = U * ((K / 16 + 18) * sums + (3 * rank + 6) * (size + z.abs()) + 2 * want.abs())
    assert bool(((out - want).abs() <= tol).all())
    assert torch.equal(out[index < 0], z[index < 0])


def test_refusals(qs):
    import torch
    B, V, K, rank, count = 3, 100, 64, 16, 2
    lg = torch.randn(B, 104, device="cuda")[:, :V]
    h = torch.randn(B, K, device="cuda").bfloat16()
    d = torch.randn(count, rank, K, device="cuda").bfloat16()
    u = torch.randn(count, V, rank, device="cuda").bfloat16()
    i = torch.zeros(B, dtype=torch.int32, device="cuda")
    s = torch.ones(count, device="cuda")
    qs.apply_adapters(lg, h, d, u, i, s)
    value = [dict(logits=lg.cpu()), dict(logits=lg[0]), dict(hidden=h.float()), dict(hidden=h[:2]),
             dict(hidden=h.cpu()), dict(hidden=h[:, :32]), dict(hidden=h.t().contiguous().t()),
             dict(down=d.float()), dict(down=d[0]), dict(down=d[:1]), dict(down=d[:, :8]),
             dict(down=d.transpose(1, 2).contiguous().transpose(1, 2)),
             dict(up=u.float()), dict(up=u[:, :50]), dict(up=u.cpu()),
             dict(up=u.transpose(1, 2).contiguous().transpose(1, 2)),
             dict(index=i.long()), dict(index=i[:2]), dict(index=i.cpu()),
             dict(scale=s.double()), dict(scale=s[:1]), dict(scale=s.cpu()),
             dict(out=torch.empty(B, V + 4, device="cuda")), dict(out=lg.cpu()),
             dict(out=torch.empty(B, 104, dtype=torch.bfloat16, device="cuda")[:, :V]),
             dict(workspace=torch.empty(1 << 12, dtype=torch.uint8)),
             dict(logits=lg.clone().requires_grad_()), dict(hidden=h.clone().requires_grad_()),
             dict(down=d.clone().requires_grad_()), dict(up=u.clone().requires_grad_()),
             dict(scale=s.clone().requires_grad_()),
             dict(out=torch.empty(B, 104, device="cuda", requires_grad=True))]
    for kw in value:
        args = dict(logits=lg, hidden=h, down=d, up=u, index=i, scale=s)
        args.update(kw)
        with pytest.raises(ValueError):
            qs.apply_adapters(**args)
    run_time = [dict(down=d[:, :4], up=u[:, :, :4]),                      # rank
                dict(hidden=h[:, :60], down=d[:, :, :60]),                # columns
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                dict(logits=torch.randn(B, 101, device="cuda")[:, :V]),   # row stride
                dict(out=lg.new_empty(B, 101)[:, :V]),
                dict(hidden=torch.randn(B, K + 1, device="cuda").bfloat16()[:, :K])]
    for kw in run_time:
        args = dict(logits=lg, hidden=h, down=d, up=u, index=i, scale=s)
        args.update(kw)
        with pytest.raises(RuntimeError):
            qs.apply_adapters(**args)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(lg, torch.ones_like(lg))
        with pytest.raises(ValueError):
            qs.apply_adapters(dual, h, d, u, i, s)
    # a graph that saved the logits sees the change in place
    leaf = torch.randn(B, 104, device="cuda", requires_grad=True)
    y = (leaf * lg.new_ones(B, 104)).exp()
    loss = (y * y.detach()).sum()
    qs.apply_adapters(y.detach()[:, :V], h, d, u, i, s)
    with pytest.raises(RuntimeError):
        loss.backward()


def test_empty_batch(qs):
    import torch
    status = qs.apply_adapters(torch.empty(0, 64, device="cuda"),
                               torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"),
                               torch.zeros(1, 8, 32, dtype=torch.bfloat16, device="cuda"),
                               torch.zeros(1, 64, 8, dtype=torch.bfloat16, device="cuda"),
                               torch.empty(0, dtype=torch.int32, device="cuda"))
    assert status.shape == (0,)


def test_offsets_past_32_bits(qs):
    """Adapters that start past 2^32 elements, and a vocabulary past 2^24 bytes a row."""
    import torch
    V, rank, count, K = 150001, 128, 240, 64
    assert (count - 1) * V * rank > 1 << 32
    up = torch.zeros(count, V, rank, dtype=torch.bfloat16, device="cuda")
    z, x, down, one, scale, _ = inputs(2, 4, V, K, rank, 2)
    up[0], up[count - 1] = to16(one[0]), to16(one[1])
    wide = torch.zeros(count, rank, K, dtype=torch.bfloat16, device="cuda")
    wide[0], wide[count - 1] = to16(down[0]), to16(down[1])
    index = np.array([count - 1, 0, 0, count - 1], np.int32)
    lg = on_gpu(z, "f32")
    qs.apply_adapters(lg, to16(x), wide, up, to(index))
    torch.cuda.synchronize()
    check(z, "f32", x, down, one, None, np.array([1, 0, 0, 1], np.int32), lg)


def test_streams_and_workspace(qs):
    """Two calls at once with scratch memory of their own; scratch memory used again."""
    import torch
    z, x, down, up, scale, index = inputs(4, 33, 30001, 512, 16, 7)
    args = (to16(x), to16(down), to16(up), to(index), to(scale))
    want = on_gpu(z, "bf16")
    qs.apply_adapters(want, *args)
    torch.cuda.synchronize()
    outs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        lg = on_gpu(z, "bf16")
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            qs.apply_adapters(lg, *args)
        outs.append(lg)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    ws = qs.adapters_workspace_for(want, 16)
    for fill in (0, 255):
        ws.fill_(fill)
        lg = on_gpu(z, "bf16")
        qs.apply_adapters(lg, *args, workspace=ws)
        few = on_gpu(z[:5], "bf16")
        qs.apply_adapters(few, args[0][:5], args[1], args[2], args[3][:5], args[4], workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(lg, want)
        check(z[:5], "bf16", x[:5], down, up, scale, index[:5], few)


def test_graph_replays(qs):
    """Captured once, replayed on other batches, hidden states and indexes."""
    import torch
    B, V, K, rank, count = 12, 5001, 128, 16, 4
    sets = [inputs(70 + k, B, V, K, rank, count) for k in range(3)]
    down, up, scale = to16(sets[0][2]), to16(sets[0][3]), to(sets[0][4])
    z, out = on_gpu(sets[0][0], "bf16"), on_gpu(sets[0][0], "bf16")
    x, index = to16(sets[0][1]), to(sets[0][5])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        qs.apply_adapters(z, x, down, up, index, scale, out=out)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        status = qs.apply_adapters(z, x, down, up, index, scale, out=out)
    for k in (1, 0, 2, 1):
        z.copy_(on_gpu(sets[k][0], "bf16"))
        x.copy_(to16(sets[k][1]))
        index.copy_(to(sets[k][5]))
        graph.replay()
        want = on_gpu(sets[k][0], "bf16")
        qs.apply_adapters(want, x, down, up, index, scale)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and not status.any()


def head(seed, V, K, group=64):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (V, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (0.5 + torch.rand(V, K // group, generator=g, device="cuda")) * (0.6 / K ** 0.5)
    return codes, scales


def test_sample_hidden_with_adapters(qs):
    """Hidden states to tokens with an adapter per row: the same as the three calls."""
    import torch
    B, V, K, rank, count = 9, 6001, 256, 16, 4
    z, x, down, up, scale, index = inputs(6, B, V, K, rank, count)
    codes, scales = head(6, V, K)
    x, down, up, index, scale = to16(x), to16(down), to16(up), to(index), to(scale)
    T = torch.full((B,), 0.9, device="cuda")
    k = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    p = torch.full((B,), 0.95, device="cuda")
    seed = torch.arange(B, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = qs.sample_hidden(x, codes, scales, None, T, k, p, dtype=dtype,
                               adapters=dict(down=down, up=up, index=index, scale=scale),
                               seed=seed, offset=torch.zeros_like(seed))
        lg = qs.head_logits(x, codes, scales, dtype=dtype)
        status = qs.apply_adapters(lg, x, down, up, index, scale)
        want = qs.sample(lg, T, k, p, seed=seed, offset=torch.zeros_like(seed))
        torch.cuda.synchronize()
        assert torch.equal(out["logits"], lg) and torch.equal(out["tokens"], want["tokens"])
        assert torch.equal(out["adapter_status"], status) and not status.any()
    plain = qs.sample_hidden(x, codes, scales, None, T, k, p, seed=seed,
                             offset=torch.zeros_like(seed))
    assert "adapter_status" not in plain
    # logits that went elsewhere would not be the ones that are drawn from
    with pytest.raises(TypeError):
        qs.sample_hidden(x, codes, scales, None, T, k, p, seed=seed,
                         offset=torch.zeros_like(seed),
                         adapters=dict(down=down, up=up, index=index, out=lg))
    index[2] = count
    out = qs.sample_hidden(x, codes, scales, None, T, k, p, seed=seed,
                           offset=torch.zeros_like(seed),
                           adapters=dict(down=down, up=up, index=index, scale=scale))
    assert out["adapter_status"].tolist() == [4 if b == 2 else 0 for b in range(B)]
    assert torch.equal(out["logits"][2], plain["logits"][2])


def test_distill_an_adapter_then_serve_it(qs):
    """The operators together, as they would be used: adapters of the 4-bit head trained
    against a teacher's top tokens, whose gradients are the formula's, and then served
    side by side in one batch, where each row gets its own adapter's logits."""
    import torch
    torch.manual_seed(0)
    B, V, K, rank = 32, 2003, 128, 8
    codes, scales = head(1, V, K, 32)
    x = torch.randn(B, K, device="cuda").bfloat16()
    base = qs.head_logits(x, codes, scales, dtype=torch.float32)
    trained = []
    for task in range(3):
        t_logits = base + 2.0 * torch.randn(B, K, device="cuda") @ torch.randn(
            K, V, device="cuda") / K ** 0.5
        t_buf = torch.empty(B, -(-V // 4) * 4, device="cuda")[:, :V]
        t_buf.copy_(t_logits)
        top = qs.token_logprobs(t_buf, torch.zeros(B, dtype=torch.int32, device="cuda"), top_n=32)
        down = (torch.randn(rank, K, device="cuda") / K ** 0.5).requires_grad_()
        up = (0.1 * torch.randn(V, rank, device="cuda")).requires_grad_()
        opt = torch.optim.SGD((down, up), lr=0.5)
        for step in range(3):
            buf = torch.zeros(B, -(-V // 4) * 4, device="cuda")
            z = buf + torch.nn.functional.pad(base + (x.float() @ down.t()) @ up.t(),
                                              (0, buf.shape[1] - V))
            z = z[:, :V]
            out = qs.distill_loss(z, top["top_ids"], top["top_logprobs"], rest=True)
            assert not out["status"].any()
            opt.zero_grad()
            out["loss"].mean().backward()
            if step == 0:
                # the same gradients from the formula in 64 bits
                st = out["state"].cpu().numpy()
                zz = z.detach().cpu().numpy()
                dz = np.stack([oracle.distill_grad_row(
                    zz[r], None, 1.0, top["top_ids"][r].cpu().numpy(),
                    top["top_logprobs"][r].cpu().numpy(), True, 1.0 / B, st[r])
                    for r in range(B)])
                h = x.float().cpu().numpy().astype(np.float64)
                d0, u0 = (t.detach().cpu().numpy().astype(np.float64) for t in (down, up))
                for got, want in ((up.grad, dz.T @ (h @ d0.T)), (down.grad, (dz @ u0).T @ h)):
                    got = got.cpu().numpy()
                    # float32 products over B rows and V tokens
                    assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)
            opt.step()
        trained.append((down.detach().bfloat16(), up.detach().bfloat16()))
    down = torch.stack([t[0] for t in trained])
    up = torch.stack([t[1] for t in trained])
    index = (torch.arange(B, device="cuda") % 4 - 1).to(torch.int32)
    served = qs.head_logits(x, codes, scales, dtype=torch.float32)
    status = qs.apply_adapters(served, x, down, up, index)
    torch.cuda.synchronize()
    assert not status.any()
    check(base.cpu().numpy(), "f32", x.float().cpu().numpy(), down.float().cpu().numpy(),
          up.float().cpu().numpy(), None, index.cpu().numpy(), served)
