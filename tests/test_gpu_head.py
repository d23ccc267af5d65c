"""qs_head_logits (through the binding) against the oracle in fp64, and the calls
that belong together: hidden states -> logits -> selection -> scores -> gradient.

Tolerance, u = 2^-24: products of a bf16 value and a code (or a code shifted by
a whole number of at most 31 + 255) are exact, so only sums round. Within a
group the terms |x| c, c <= 32 + |zero - 8| the largest factor used, pass at
most 160 additions; group sums pass at most K / 32 + 16 more. So an element is
off by at most u (160 + K / 32 + 16) sum_g |s_g| c_g sum |x|, and by half a step
of the output type.
"""

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def qs():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_sampling_vocabs_amd as qs
    qs.load()
    return qs


def make(seed, B, V, K, group, zeros, scale, positive=False):
    import torch
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (B, K)).astype(np.float32)
    if positive:
        x = np.abs(x) + 0.5
    x = torch.from_numpy(x).to(torch.bfloat16)
    codes = torch.from_numpy(rng.integers(0, 256, (V, K // 2)).astype(np.uint8))
    s = torch.from_numpy(rng.uniform(-1, 1, (V, K // group)).astype(np.float32))
    s = s.to(torch.bfloat16) if scale == "bf16" else s
    z = torch.from_numpy(rng.integers(0, 16, (V, K // group)).astype(np.uint8)) if zeros else None
    return x, codes, s, z


def check(x, codes, s, z, group, got, out):
    import torch
    xf = x.float().numpy().astype(np.float64)
    sf = s.float().numpy().astype(np.float64)
    zn = None if z is None else z.numpy()
    K = xf.shape[1]
    want = xf @ oracle.head_weights(codes.numpy(), sf, zn, group).T
    c = 32.0 + (0.0 if zn is None else np.abs(zn.astype(np.float64) - 8))
    tol = U * (176 + K / 32) * (np.abs(xf).reshape(xf.shape[0], -1, group).sum(2)
                                @ (np.abs(sf) * c).T)
    half = 2.0 ** -24 if out == "f32" else 2.0 ** -8
    g = got.float().cpu().numpy().astype(np.float64)
    bad = np.abs(g - want) > tol * 1.01 + half * np.abs(want) * 1.01
    assert not bad.any(), (np.argwhere(bad)[:4], g[bad][:4], want[bad][:4])
    assert got.dtype == (torch.float32 if out == "f32" else torch.bfloat16)


CASES = [
    # B, V, K, group, zeros, scale, out
    (1, 1, 32, 32, False, "bf16", "f32"),
    (1, 15, 64, 64, True, "f32", "f32"),
    (1, 17, 128, 128, False, "bf16", "bf16"),
    (2, 1000, 96, 32, True, "bf16", "f32"),
    (3, 333, 160, 32, False, "f32", "bf16"),
    (5, 1009, 320, 64, True, "f32", "f32"),
    (7, 513, 384, 128, True, "bf16", "f32"),
    (8, 4099, 1024, 128, False, "f32", "f32"),
    (9, 777, 2048, 64, False, "bf16", "f32"),
    (15, 2001, 4096, 32, True, "f32", "f32"),
    (16, 2048, 4096, 128, True, "bf16", "bf16"),
    (17, 1111, 4096, 64, True, "bf16", "f32"),
    (31, 640, 8192, 128, False, "f32", "f32"),
    (32, 300, 8192, 32, True, "bf16", "f32"),
    (33, 515, 1056, 32, True, "bf16", "f32"),
    (47, 2500, 4160, 64, False, "f32", "f32"),
    (64, 1237, 8192, 64, True, "f32", "f32"),
    (65, 129, 512, 128, False, "bf16", "f32"),
    (130, 65, 1280, 128, True, "f32", "f32"),
    (1, 300, 65536, 128, True, "bf16", "f32"),
    (20, 40, 32800, 32, False, "bf16", "f32"),
    (4, 70001, 256, 64, True, "bf16", "f32"),
    (1, 40000, 1024, 32, True, "bf16", "bf16"),
    # 17 to 32 rows in registers (one, two and four steps a slice) and through LDS
    (32, 300, 96, 32, True, "bf16", "f32"),
    (31, 33000, 2176, 64, False, "bf16", "f32"),
    (18, 9001, 1280, 128, True, "f32", "bf16"),
    (29, 4003, 3968, 128, False, "bf16", "f32"),
    (24, 20001, 1024, 64, True, "bf16", "f32"),
    (16, 2100, 8192, 32, True, "bf16", "f32"),
    # 16 slices of k: full, nearly full, a last one empty
    (16, 3001, 8192, 64, True, "f32", "f32"),
    (3, 2100, 5152, 32, True, "bf16", "f32"),
    (9, 24001, 6272, 128, True, "bf16", "bf16"),
    (2, 30001, 5248, 128, False, "f32", "f32"),
    (5, 101, 4224, 32, False, "bf16", "f32"),
    (1, 21001, 7168, 32, True, "f32", "bf16"),
    # blocks of 16 rows in registers, the last one short, and beside them through LDS
    (64, 1003, 8192, 128, False, "bf16", "f32"),
    (49, 2001, 4096, 64, True, "bf16", "f32"),
    (33, 4099, 1024, 32, True, "f32", "bf16"),
    (18, 1999, 2048, 128, True, "bf16", "f32"),
    (23, 9001, 6144, 64, False, "bf16", "f32"),
    (64, 9001, 2048, 64, True, "bf16", "f32"),
    (40, 15001, 8192, 128, False, "f32", "f32"),
    (30, 15001, 8192, 32, True, "bf16", "f32"),
    (66, 1001, 4096, 64, True, "bf16", "f32"),
    # 6 to 16 rows through LDS; one to five tiles a wave; fewer groups than a lane
    # of scales holds, and groups that end inside a block of them
    (6, 20489, 384, 64, True, "bf16", "f32"),
    (16, 24001, 1056, 32, True, "f32", "f32"),
    (13, 70003, 640, 128, False, "bf16", "bf16"),
    (64, 100001, 160, 32, True, "bf16", "f32"),
    (40, 131077, 384, 128, True, "f32", "bf16"),
    (33, 163841, 320, 64, False, "bf16", "bf16"),
    (50, 150000, 96, 32, False, "f32", "f32"),
    (20, 140001, 128, 128, True, "bf16", "f32"),
    (64, 170003, 32, 32, True, "f32", "f32"),
    (17, 40003, 832, 32, True, "bf16", "f32"),
    (64, 17000, 4480, 128, True, "bf16", "f32"),
    (34, 50001, 704, 64, True, "f32", "bf16"),
    (64, 3, 32, 32, True, "bf16", "f32"),
    (40, 1, 64, 64, True, "f32", "f32"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_oracle(qs, case):
    import torch
    B, V, K, group, zeros, scale, out = case
    print("head", case, flush=True)
    x, codes, s, z = make(K + B, B, V, K, group, zeros, scale)
    d = torch.float32 if out == "f32" else torch.bfloat16
    got = qs.head_logits(x.cuda(), codes.cuda(), s.cuda(), None if z is None else z.cuda(), dtype=d)
    torch.cuda.synchronize()
    check(x, codes, s, z, group, got, out)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("B", [1, 12, 30, 64])
def test_nothing_left_from_before(qs, B, group):
    """Groups past the row's end, in rows of one short chunk and of several, do not
    see what an earlier call left on chip: here NaN and infinite scales."""
    import torch
    print(f"head leftovers B={B} group={group}", flush=True)
    V = 24001
    x, codes, s, z = (t.cuda() for t in make(3, B, V, 512, group, True, "f32"))
    for K in (group, 256 + group, 384):
        if K % group:
            continue
        for fill in (float("nan"), float("inf")):
            qs.head_logits(x, codes, torch.full_like(s, fill), z, dtype=torch.float32)
            got = qs.head_logits(x[:, :K], codes[:, :K // 2], s[:, :K // group], z[:, :K // group],
                                 dtype=torch.float32)
            torch.cuda.synchronize()
            check(x[:, :K].cpu(), codes[:, :K // 2].cpu(), s[:, :K // group].cpu(),
                  z[:, :K // group].cpu(), group, got, "f32")


@pytest.mark.parametrize("B", [1, 6, 20, 64])
def test_strides_and_padding(qs, B):
    """Row strides of every operand; rows and columns around the result stay."""
    import torch
    print(f"head strides B={B}", flush=True)
    V, K, group = 1003, 1152, 64
    x, codes, s, z = make(B, B, V, K, group, True, "f32")
    xs = torch.full((B, K + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    xs[:, :K] = x.cuda()
    cs = torch.full((V, K // 2 + 48), 255, dtype=torch.uint8, device="cuda")
    cs[:, :K // 2] = codes.cuda()
    ss = torch.full((V, K // group + 3), float("nan"), device="cuda")
    ss[:, :K // group] = s.cuda()
    zs = torch.full((V, K // group + 5), 255, dtype=torch.uint8, device="cuda")
    zs[:, :K // group] = z.cuda()
    buf = torch.full((B + 2, 1080), 5.0, device="cuda")
    out = qs.head_logits(xs[:, :K], cs[:, :K // 2], ss[:, :K // group], zs[:, :K // group],
                         out=buf[1:B + 1, 4:4 + V])
    torch.cuda.synchronize()
    check(x, codes, s, z, group, out, "f32")
    assert (buf[0] == 5).all() and (buf[B + 1] == 5).all()
    assert (buf[1:B + 1, :4] == 5).all() and (buf[1:B + 1, 4 + V:] == 5).all()
    plain = qs.head_logits(x.cuda(), codes.cuda(), s.cuda(), z.cuda(), dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(plain, out)


@pytest.mark.parametrize("B", [2, 20, 40])
def test_offsets_past_32_bits(qs, B):
    """Rows of codes and logits that lie 2^32 bytes and more into their buffers,
    in every kernel, at strides that a row of 4-bit weights can have."""
    import torch
    print(f"head offsets B={B}", flush=True)
    V, K, group, stride = 70003, 128, 64, 65536
    x, codes, s, z = make(B, B, V, K, group, True, "f32")
    cs = torch.empty((V, stride), dtype=torch.uint8, device="cuda")[:, :K // 2]
    cs.copy_(codes)
    rows = torch.empty((B, 1 << 29), dtype=torch.float32, device="cuda")[:, :V]
    got = qs.head_logits(x.cuda(), cs, s.cuda(), z.cuda(), out=rows)
    torch.cuda.synchronize()
    check(x, codes, s, z, group, got, "f32")


@pytest.mark.parametrize("B", [1, 16, 64])
def test_one_sided_values(qs, B):
    """Hidden values of one sign (the codes' offset does not cancel by chance),
    zero points far from 8, codes at both ends."""
    import torch
    print(f"head one-sided B={B}", flush=True)
    x, codes, s, z = make(9, B, 257, 4096, 128, True, "f32", positive=True)
    z = torch.where(z > 7, 255, 0).to(torch.uint8)
    codes[:100] = 0
    codes[100:200] = 255
    got = qs.head_logits(x.cuda(), codes.cuda(), s.cuda(), z.cuda(), dtype=torch.float32)
    torch.cuda.synchronize()
    check(x, codes, s, z, 128, got, "f32")


def test_non_finite_hidden_rows(qs):
    """An infinity or a NaN stays in its row, and there no logit is finite."""
    import torch
    for B in (4, 40):
        x, codes, s, z = make(3, B, 400, 512, 32, True, "f32")
        x[1, 5] = float("inf")
        x[2, 511] = float("nan")
        got = qs.head_logits(x.cuda(), codes.cuda(), s.cuda(), z.cuda(), dtype=torch.float32)
        torch.cuda.synchronize()
        lost = ~torch.isfinite(got).cpu()
        assert lost[1].all() and lost[2].all() and lost.sum() == 800
        assert torch.isnan(got[2]).all()
        keep = [r for r in range(B) if r not in (1, 2)]
        check(x[keep], codes, s, z, 32, got[keep], "f32")


@pytest.mark.parametrize("B", [1, 12, 48])
def test_same_bits(qs, B):
    """The same call twice, and rows on their own or in a batch with other rows."""
    import torch
    x, codes, s, z = (t.cuda() for t in make(4, B, 3001, 2048, 64, True, "bf16"))
    a = qs.head_logits(x, codes, s, z, dtype=torch.float32)
    b = qs.head_logits(x, codes, s, z, dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_refusals(qs):
    import torch
    x, codes, s, z = (t.cuda() for t in make(1, 2, 64, 256, 64, True, "f32"))
    for kw in (dict(hidden=x.float()), dict(hidden=x.cpu()), dict(hidden=x[0]),
               dict(hidden=x[:, :128]), dict(codes=codes.to(torch.int32)), dict(codes=codes[:, :64]),
               dict(codes=codes.cpu()), dict(scales=s[:60]), dict(scales=s[:, :3]),
               dict(scales=s[:, :1]), dict(zeros=z[:, :2]), dict(zeros=z.to(torch.int32)),
               dict(zeros=z.cpu()), dict(out=torch.zeros(2, 63, device="cuda")),
               dict(out=torch.zeros(2, 64), dtype=torch.float32),
               dict(out=torch.zeros(2, 64, device="cuda"), dtype=torch.bfloat16),
               dict(hidden=x.clone().requires_grad_())):
        a = dict(hidden=x, codes=codes, scales=s, zeros=z) | kw
        with pytest.raises(ValueError):
            qs.head_logits(a.pop("hidden"), a.pop("codes"), a.pop("scales"), a.pop("zeros"), **a)
    with pytest.raises(TypeError):
        qs.head_logits(x, codes, s.half(), z)
    with pytest.raises(RuntimeError):      # rows of logits that do not start 16-byte aligned
        qs.head_logits(x, codes, s, z, out=torch.zeros(2, 65, device="cuda")[:, :64])
    with pytest.raises(RuntimeError):      # rows of codes that do not start 16-byte aligned
        qs.head_logits(x, torch.zeros(64, 136, dtype=torch.uint8, device="cuda")[:, :128], s, z)
    assert qs.head_logits(x[:0], codes, s, z).shape == (0, 64)


# --------------------------------------------------------------------------
# Together

def chain(qs, x, codes, s, z, par, tok2):
    """One decode step and its training signal, as a rollout runs them."""
    import torch
    out = qs.sample_hidden(x, codes, s, z, par["T"], par["k"], par["p"], par["bm"],
                           uniforms=par["u"], logprobs=True, logits=par.get("buf"))
    lg = out["logits"]
    sc = qs.token_logprobs(lg, torch.stack((out["tokens"], tok2), 1), temperature=par["T"],
                           bitmask=par["bm"], entropy=True, top_n=5, workspace=par.get("ws"))
    grad = qs.token_logprobs_backward(
        lg, torch.stack((out["tokens"], tok2), 1), sc["row_max"], sc["log_sum"], sc["status"],
        par["gl"], temperature=par["T"], bitmask=par["bm"], entropy=sc["entropy"],
        grad_entropy=par["gH"])
    return {"tokens": out["tokens"], "sampled": out["logprobs"], "status": out["status"],
            "logits": lg, "grad": grad, **{"score_" + k: v for k, v in sc.items()}}


def chain_inputs(qs, seed=2, B=12, V=5003, K=1024):
    import torch
    rng = np.random.default_rng(seed)
    x, codes, s, z = (t.cuda() for t in make(seed, B, V, K, 128, True, "bf16"))
    s *= 0.05
    bm = rng.integers(0, 2 ** 32, (B, -(-V // 32)), dtype=np.uint32).view(np.int32)
    par = dict(T=torch.full((B,), 0.8, device="cuda"),
               k=torch.zeros(B, dtype=torch.int32, device="cuda"),
               p=torch.ones(B, device="cuda"), bm=torch.from_numpy(bm).cuda(),
               u=torch.from_numpy(rng.random(B)).cuda(),
               gl=torch.from_numpy(rng.normal(0, 1, (B, 2)).astype(np.float32)).cuda(),
               gH=torch.from_numpy(rng.normal(0, 1, B).astype(np.float32)).cuda())
    tok2 = torch.from_numpy(rng.integers(0, V, B).astype(np.int32)).cuda()
    return x, codes, s, z, par, tok2


def bits(t):
    import torch
    return t.contiguous().view({4: torch.int32, 2: torch.int16}[t.element_size()])


def test_decode_step_and_gradient(qs):
    """The operators one after another, each against the oracle on what the one
    before it gave. With top-k and top-p off, the scores of the drawn tokens
    are the log-probabilities that the draw reports. Scores are held to 2^-24
    times 140 additions, 4 |ln p| (below 25 for what is drawn) and 16 more;
    gradients to 2^-24 (4 |a| + 24) times the sum of the slots' gradients, where
    p |a| stays below 1, and half a bf16 step."""
    import torch
    x, codes, s, z, par, tok2 = chain_inputs(qs)
    got = chain(qs, x, codes, s, z, par, tok2)
    torch.cuda.synchronize()
    check(x.cpu(), codes.cpu(), s.cpu(), z.cpu(), 128, got["logits"], "bf16")
    lg = got["logits"].float().cpu().numpy().astype(np.float64)
    words = par["bm"].cpu().numpy().view(np.uint32)
    for r in range(lg.shape[0]):
        legal = oracle.legal_from_bitmask(words[r], lg.shape[1])
        t = [int(got["tokens"][r]), int(tok2[r])]
        want = oracle.score_row(lg[r], legal, 0.8, t, 5)
        assert got["status"][r] == 0 and want["status"] == 0 and legal[t[0]]
        lps = got["score_logprobs"][r].cpu().numpy()
        assert abs(lps[0] - want["logprobs"][0]) <= 2e-5
        assert abs(float(got["sampled"][r]) - lps[0]) <= 2e-5
        assert np.array_equal(got["score_top_ids"][r].cpu().numpy(), want["top_ids"])
        H = float(got["score_entropy"][r])
        g = oracle.grad_row(lg[r], legal, np.float32(0.8), t, par["gl"][r].cpu().numpy(),
                            float(par["gH"][r]), float(got["score_row_max"][r]),
                            float(got["score_log_sum"][r]), H)
        d = np.abs(got["grad"][r].float().cpu().numpy() - g)
        assert (d <= 2.0 ** -8 * 1.01 * np.abs(g) + 1e-5).all(), d.max()


def test_two_streams(qs):
    """Chains on two streams at once give what they give one after another."""
    import torch
    ins = [chain_inputs(qs, seed=k, B=3 + 10 * k, V=40000 + k) for k in (1, 2)]
    want = [chain(qs, *i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(3):
        got = []
        for st, i in zip(streams, ins):
            with torch.cuda.stream(st):
                got.append(chain(qs, *i))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for k in b:
                assert torch.equal(bits(a[k]), bits(b[k])), k


def test_captured_and_replayed(qs):
    """A captured chain, replayed with eager work and new inputs between."""
    import torch
    x, codes, s, z, par, tok2 = chain_inputs(qs, seed=6, B=5, V=60001)
    par["ws"] = qs.token_logprobs_workspace_for(
        torch.empty(5, 60001 + 7, dtype=torch.bfloat16, device="cuda")[:, :60001], 5)
    cs = torch.cuda.Stream()
    cs.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cs):
        chain(qs, x, codes, s, z, par, tok2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cs):
        out = chain(qs, x, codes, s, z, par, tok2)
    torch.cuda.synchronize()
    for k in range(4):
        x.copy_(torch.randn(x.shape, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.stream(cs):
            g.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in out.items()}
        want = chain(qs, x, codes, s, z, dict(par, ws=None), tok2)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(bits(got[n]), bits(want[n])), (k, n)


def long_chain(qs, seed, B, V):
    """chain_inputs for rows of several parts, with scratch memory of their own."""
    import torch
    x, codes, s, z, par, tok2 = chain_inputs(qs, seed=seed, B=B, V=V, K=512)
    par["ws"] = qs.token_logprobs_workspace_for(
        torch.empty((B, -(-V // 8) * 8), dtype=torch.bfloat16, device="cuda")[:, :V], 5)
    assert par["ws"] is not None
    return x, codes, s, z, par, tok2


def test_two_streams_long_rows(qs):
    """test_two_streams with rows whose parts pass through scratch memory, the
    caller's and the call's own."""
    import torch
    ins = [long_chain(qs, k, 3 + 10 * k, 131072 + k) for k in (1, 2)]
    want = [chain(qs, *i[:4], dict(i[4], ws=None), i[5]) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for own in (False, True, False):
        got = []
        for st, i in zip(streams, ins):
            with torch.cuda.stream(st):
                got.append(chain(qs, *i[:4], dict(i[4], ws=None) if own else i[4], i[5]))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for k in b:
                assert torch.equal(bits(a[k]), bits(b[k])), k


@pytest.mark.parametrize("own", [False, True])
def test_captured_and_replayed_long_rows(qs, own):
    """test_captured_and_replayed with rows of several parts; two graphs with the
    caller's scratch memory each, or with the graph's own."""
    import torch
    ins = [long_chain(qs, 5 + k, 5 + k, 131077 + k) for k in (0, 1)]
    if own:
        for i in ins:
            i[4]["ws"] = None
    cs = torch.cuda.Stream()
    cs.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cs):
        for i in ins:
            chain(qs, *i)
    torch.cuda.synchronize()
    graphs = []
    for i in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=cs):
            out = chain(qs, *i)
        graphs.append((g, out))
    torch.cuda.synchronize()
    for k in range(4):
        for i in ins:
            i[0].copy_(torch.randn(i[0].shape, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.stream(cs):
            for g, _ in graphs:
                g.replay()
        torch.cuda.synchronize()
        for i, (_, out) in zip(ins, graphs):
            got = {n: v.clone() for n, v in out.items()}
            want = chain(qs, *i[:4], dict(i[4], ws=None), i[5])
            torch.cuda.synchronize()
            for n in want:
                assert torch.equal(bits(got[n]), bits(want[n])), (k, n)


@pytest.mark.parametrize("B", [1, 8, 20, 40])
def test_most_vocabulary_rows(qs, B):
    """2^24 vocabulary rows, the most a call takes: every logit of some rows' tiles,
    the first and the last among them."""
    import torch
    print(f"head most vocabulary rows B={B}", flush=True)
    V, K = 1 << 24, 32
    x, codes, s, z = make(B, B, 4096, K, 32, True, "bf16")
    many = V // 4096
    # every block of 4096 rows of weights is the same but for its scale, a power of two
    power = torch.exp2((torch.arange(many, device="cuda") % 7).float()).repeat_interleave(4096)
    scales = (s.cuda().repeat(many, 1).float() * power[:, None]).bfloat16()
    got = qs.head_logits(x.cuda(), codes.cuda().repeat(many, 1), scales, z.cuda().repeat(many, 1))
    torch.cuda.synchronize()
    blocks = got.view(B, many, 4096)
    check(x, codes, s, z, 32, blocks[:, 0], "bf16")
    assert torch.equal(blocks.float(), blocks[:, :1].float()
                       * power.view(many, 4096)[None])


def test_most_rows(qs):
    """2^20 hidden rows, the most a call takes, and the first count past them."""
    import torch
    print("head most rows", flush=True)
    B, V, K = 1 << 20, 19, 64
    x, codes, s, z = make(7, B, V, K, 64, True, "f32")
    got = qs.head_logits(x.cuda(), codes.cuda(), s.cuda(), z.cuda(), dtype=torch.float32)
    torch.cuda.synchronize()
    check(x, codes, s, z, 64, got, "f32")
    with pytest.raises(RuntimeError):
        qs.head_logits(torch.zeros(B + 1, K, dtype=torch.bfloat16, device="cuda"), codes.cuda(),
                       s.cuda(), z.cuda())


def test_empty_batch_of_hidden_states(qs):
    import torch
    x, codes, s, z = (t.cuda() for t in make(1, 2, 64, 256, 64, True, "f32"))
    none = torch.zeros(0, device="cuda")
    out = qs.sample_hidden(x[:0], codes, s, z, none, none.int(), none,
                           uniforms=none.double())
    assert out["logits"].shape == (0, 64) and out["tokens"].shape == (0,)
