"""Beam selection on the GPU against the plain 64-bit reference.

Tolerance of a score, from the kernel's arithmetic.  Its own rounding to fp32
is at most half a step: 2^-24 |score|.  The row sum S = sum exp(l - ref) carries,
relative to S: ex2.approx 2^-22; the fp32 sum of the up to 32 elements of a
lane's tile, 17 * 2^-24; and in the exponent d = l - ref one rounding of l c - E
(2^-24 relative) and that of c = log2 e in fp32 (2^-26), which weigh 1.25 * 2^-24
sum p |d|.  The reference lies up to 8 above the largest logit, and the rest of
|d| = -log p - log S weighs at most the entropy, log V <= 16.7: 1.25 * 2^-24 *
24.7.  Together below 2.4e-7 + 1.02e-6 + 1.85e-6 < 4e-6, which log S carries as
an absolute error.
Two candidates of different beams whose values are more than twice that apart
are in the reference's order; candidates of one beam always are."""
import numpy as np
import pytest

import decode_reference as ref
from gpu_util import host, require_cuda

pytestmark = pytest.mark.gpu
EPS = 4e-6


@pytest.fixture(scope="module")
def torch_():
    return require_cuda()


@pytest.fixture(scope="module")
def ver(torch_):
    import speculative_decoding_draft_decode_b200 as sd
    return sd.Verifier(torch_.device("cuda", 0))


def rows_of(torch, x, dtype, pad=0, offset=0):
    """x [B, W, V] on the device as `dtype`, rows `pad` elements apart and the
    first `offset` elements into its allocation; and the stored values."""
    B, W, V = x.shape
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    flat = torch.zeros(offset + B * W * (V + pad), dtype=dt, device="cuda")
    t = flat[offset:].view(B, W, V + pad)[..., :V]
    t.copy_(torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dt))
    return t, t.cpu().double().numpy()


def check(torch, ver, x, scores, K, dtype="f32", pad=0, offset=0, finished=None, eos=0, **kw):
    t, stored = rows_of(torch, x, dtype, pad, offset)
    s = torch.from_numpy(scores.astype(np.float32)).cuda()
    f = None if finished is None else torch.from_numpy(finished.astype(np.int32)).cuda()
    got = [host(a) for a in ver.beam_select(t, s, K, finished=f, eos_token=eos, **kw)]
    compare(got, stored, scores.astype(np.float32).astype(np.float64), K, finished, eos)
    return got


def compare(got, stored, scores, K, finished=None, eos=0):
    V = stored.shape[2]
    e_s, e_p, e_t, values = ref.beam_select(stored, scores, K, finished, eos)
    g_s, g_p, g_t = got
    assert np.array_equal(np.isnan(g_s), np.isnan(e_s))
    for b in range(len(g_s)):
        if np.isnan(e_s[b]).any():
            assert (g_p[b] == -1).all() and (g_t[b] == -1).all()
            continue
        real = e_s[b] > -np.inf
        assert np.array_equal(g_s[b][~real], e_s[b][~real]) and (g_p[b][~real] == -1).all() and \
            (g_t[b][~real] == -1).all()
        n = int(real.sum())
        tol = 2.0**-24 * np.abs(e_s[b][:n]) + EPS
        assert (np.abs(g_s[b][:n] - e_s[b][:n]) <= tol).all()
        flat = g_p[b][:n].astype(np.int64) * V + g_t[b][:n]
        assert len(set(flat.tolist())) == n and (g_p[b][:n] >= 0).all() and (g_t[b][:n] >= 0).all()
        # each place holds the reference's candidate, or one of another beam within 2 EPS of it
        want = e_p[b][:n].astype(np.int64) * V + e_t[b][:n]
        for j in np.nonzero(flat != want)[0]:
            assert g_p[b][j] != e_p[b][j] or (g_p[b] != e_p[b]).any()
            assert abs(values[b][flat[j]] - e_s[b][j]) <= 2 * EPS
        for w in set(g_p[b][:n].tolist()):  # one beam's candidates: its best, in the exact order
            mine = g_t[b][:n][g_p[b][:n] == w]
            row = values[b][w * V:(w + 1) * V]
            if finished is None or not finished[b, w]:
                assert np.array_equal(mine, np.argsort(-row, kind="stable")[:len(mine)])
    return e_s, e_p, e_t


def logits(rng, B, W, V, scale=2.0):
    x = rng.standard_normal((B, W, V)).astype(np.float32) * scale
    x[np.arange(B)[:, None], np.arange(W)[None], rng.integers(0, V, (B, W))] += 8.0
    return x


def beam_scores(rng, B, W):
    return -np.cumsum(rng.random((B, W)) * 1.5, 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,W,K,V", [(1, 1, 1, 1), (3, 2, 4, 1), (2, 3, 5, 7), (4, 4, 4, 33), (2, 8, 32, 100), (4, 4, 4, 1000),
                                     (3, 5, 10, 4099), (2, 2, 32, 16387), (2, 32, 32, 515), (2, 3, 8, 40001),
                                     (1, 2, 16, 151935)])
def test_sizes(torch_, ver, dtype, B, W, K, V):
    rng = np.random.default_rng(B * 1000 + V)
    check(torch_, ver, logits(rng, B, W, V), beam_scores(rng, B, W), K, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (8, 0), (3, 1), (0, 3), (5, 7)])
def test_strides_and_alignment(torch_, ver, dtype, pad, offset):
    rng = np.random.default_rng(pad * 10 + offset)
    for V in (9, 2051, 20000):
        check(torch_, ver, logits(rng, 2, 3, V), beam_scores(rng, 2, 3), 6, dtype, pad, offset)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masks(torch_, ver, dtype):
    """Grammar masks (-inf), the type's lowest value, rows that nothing is left of."""
    rng = np.random.default_rng(7)
    low = -3.3895313892515355e38 if dtype == "bf16" else float(np.finfo(np.float32).min)
    for V in (60, 5000, 33000):
        x = logits(rng, 4, 3, V)
        x[0][:, rng.random(V) < 0.9] = -np.inf
        x[1] = np.where(rng.random((3, V)) < 0.999, low, x[1])
        x[2, 0] = -np.inf                       # nothing left of one row
        x[2, 1] = low                           # everything masked with the lowest value
        x[3] = -np.inf                          # nothing left of a request
        x[2, 2, 5:] = -np.inf                   # fewer candidates than asked for
        check(torch_, ver, x, beam_scores(rng, 4, 3), 12, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 8, 32])
def test_equal_values(torch_, ver, dtype, K):
    """Ties go to the lowest w V + v: rows of one value, of few values, of
    signed zeros; more ties than any buffer holds."""
    rng = np.random.default_rng(3)
    for V in (40, 1000, 3000, 20480):
        x = np.zeros((5, 4, V), np.float32)
        x[1] = rng.integers(0, 2, (4, V))
        x[2] = np.where(rng.random((4, V)) < 0.5, -0.0, 0.0)
        x[3] = 1.5
        x[3, :, V // 2:] = 2.5
        x[4] = np.round(rng.standard_normal((4, V)))
        check(torch_, ver, x, np.zeros((5, 4)) - np.arange(4) * 0.25, K, dtype)
    # every beam alike and aligned alike: candidates of all beams tie
    x = np.repeat(rng.standard_normal((1, 1, 4096)).astype(np.float32), 8, 1)
    s, p, t = check(torch_, ver, x, np.zeros((1, 8)) - 1.0, K, dtype)
    assert (p[0][:min(K, 8)] == np.arange(min(K, 8))).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W,V", [(2, 700), (2, 9000), (3, 40003), (3, 400003)])
def test_logits_that_differ_less_than_their_values(torch_, ver, dtype, W, V):
    """Two logits of a row whose values are one number in 64 bits (logits next
    to zero, or scores so low that no logit shows beside them) are still in the
    logits' order."""
    torch = torch_
    rng = np.random.default_rng(29)
    x = rng.standard_normal((5, W, V)).astype(np.float32)
    x[0] *= 1e-18
    x[1] *= 1e-30
    x[2, :, V // 2:] *= 1e-20
    x[2, :, :V // 2] = -1.0
    x[0, :, 5], x[0, :, 3] = 0.0, -0.0
    s = np.full((5, W), -1.0, np.float32) - np.arange(W, dtype=np.float32) * 0.125
    s[3] = -1e30
    s[4] = np.finfo(np.float32).min
    t, stored = rows_of(torch, x, dtype)
    for K in (1, 6, 20, 32):
        _, p, tok = (host(a) for a in ver.beam_select(t, torch.from_numpy(s).cuda(), K))
        for b in range(5):
            assert (p[b] >= 0).all() and len(set(zip(p[b].tolist(), tok[b].tolist()))) == K
            for w in set(p[b].tolist()):
                mine = tok[b][p[b] == w]
                assert np.array_equal(mine, np.argsort(-stored[b, w], kind="stable")[:len(mine)])


def test_ties_over_many_chunks(torch_, ver):
    """32 beams of one value over several chunks: more candidates at the bound
    than the merge holds."""
    x = np.zeros((2, 32, 50000), np.float32)
    x[1] = np.round(np.random.default_rng(0).standard_normal((32, 50000)) * 0.6)
    check(torch_, ver, x, np.zeros((2, 32)) - np.arange(32) * 0.125, 32)


def test_beams_without_hypothesis_and_finished(torch_, ver):
    rng = np.random.default_rng(11)
    for V, K in ((100, 8), (30000, 20)):
        B, W = 6, 5
        x = logits(rng, B, W, V)
        s = beam_scores(rng, B, W)
        fin = (rng.random((B, W)) < 0.4).astype(np.int32)
        s[0, 1:] = -np.inf      # the first step of a search
        s[1] = -np.inf          # no hypothesis at all
        fin[2] = 1              # all have ended: W candidates
        fin[0] = 0
        fin[1] = 1
        x[2] = np.nan           # rows of finished beams are not read
        x[0, 1:] = np.inf       # nor those without a hypothesis
        check(torch_, ver, x, s, K, finished=fin, eos=7)
        check(torch_, ver, x, np.where(fin, -np.inf, s), K)


def test_undefined_requests(torch_, ver):
    rng = np.random.default_rng(13)
    for V in (50, 9001):
        x = logits(rng, 6, 3, V)
        s = beam_scores(rng, 6, 3)
        x[0, 1, V // 2] = np.nan
        x[1, 2, V - 1] = np.inf
        s[2, 0] = np.nan
        s[3, 1] = np.inf
        x[4, 0] = np.nan
        check(torch_, ver, x, s, 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_crowded_tiles(torch_, ver, dtype):
    """Real vocabularies are not shuffled: the likely tokens stand together, so
    one tile holds many more candidates than K, or all of them; and rows whose
    logits are far from zero."""
    rng = np.random.default_rng(17)
    for V, K in ((6000, 8), (40000, 32)):
        x = rng.standard_normal((4, 3, V)).astype(np.float32)
        x[0] += np.linspace(30, 0, V)[None]          # falling with the index
        x[1, :, 1000:2100] += 9.0                    # one crowded stretch
        x[2] += 900.0
        x[3] = x[3] * 1e-3 - 5e4
        check(torch_, ver, x, beam_scores(rng, 4, 3), K, dtype)


def test_huge_logits(torch_, ver):
    """Values near the ends of fp32, where the reference times log2 e overflows."""
    rng = np.random.default_rng(18)
    x = rng.standard_normal((3, 2, 9000)).astype(np.float32)
    x[0] = x[0] * 2e37
    x[1] = -3.0e38 + np.abs(x[1]) * 1e37
    x[2, 0] = np.float32(2.0e37)
    x[2, 1] = -np.float32(2.0e37)
    check(torch_, ver, x, beam_scores(rng, 3, 2), 6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-1e6, -1e8, -1e9, -2.5e9, -1e10, -1e15, -1e20, -1e30, -1e36])
def test_masks_of_finite_values(torch_, ver, dtype, low):
    """Masks of a large finite value: stretches of whole tiles (and of whole
    segments of them) at the start, in the middle and at the end of a row, whole
    rows, and scattered tokens; with one launch, with mended sums and without."""
    rng = np.random.default_rng(23)
    for W, V in ((2, 3000), (3, 7000), (3, 30000), (2, 41001)):
        x = logits(rng, 6, W, V)
        x[0, :, :V // 2] = low
        x[1, :, V // 4:3 * V // 4] = low
        x[2, :, V // 3:] = low
        x[3] = np.where(rng.random((W, V)) < 0.7, low, x[3])
        x[4, 0] = low                       # nothing else in one row
        x[5] = low                          # nor in a request
        x[5, 1, 7:9] = low * 1.5
        check(torch_, ver, x, beam_scores(rng, 6, W), 6, dtype)
        check(torch_, ver, x, beam_scores(rng, 6, W), 24, dtype, pad=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at", [3e4, 65530.0, 65536.0, 7e4, 9.9e5, 1.1e6, 1e8, 1e9, 2.5e9, 1e10, 1e15, 1e20, 1e30, 1e36, 1.01e37])
def test_far_references(torch_, ver, dtype, at):
    """Rows around any finite value, of either sign: close to it, spread around
    it, of nothing but it, and in stretches of it among ordinary logits.  The
    tolerance is the same: the rounding of E is part of the reference, and from
    2^16 on d = l - ref is exact where its term does not vanish (l within a factor
    2 of ref), which leaves the one rounding of d c."""
    rng = np.random.default_rng(24)
    for W, V in ((2, 3000), (3, 7000), (3, 30000)):
        x = rng.standard_normal((6, W, V)) * 2.0
        for b, v in enumerate((at, -at)):
            x[b] = v + x[b]
            x[2 + b] = v * (1.0 + 1e-2 * x[2 + b])
        x[4, :, V // 2:] = at
        x[5, 0] = -at
        x[5, 1] = at
        check(torch_, ver, x.astype(np.float32), beam_scores(rng, 6, W), 7, dtype)


def test_large_vocabulary(torch_, ver):
    """2^20 + 3 tokens: a row's partials span many chunks."""
    torch = torch_
    g = torch.Generator("cuda")
    g.manual_seed(1)
    x = torch.randn((1, 2, (1 << 20) + 3), generator=g, device="cuda")
    s = torch.tensor([[-0.5, -0.7]], device="cuda")
    got = [host(a) for a in ver.beam_select(x, s, 9)]
    compare(got, x.cpu().double().numpy(), s.cpu().double().numpy(), 9)


def test_out_streams_and_graphs(torch_, ver):
    """Given outputs, another stream, and a captured call replayed on new
    inputs, with larger calls (which grow the workspace) in between."""
    import speculative_decoding_draft_decode_b200 as sd
    torch = torch_
    rng = np.random.default_rng(5)
    mine = sd.Verifier(torch.device("cuda", 0))
    B, W, K, V = 3, 4, 6, 5000
    xs = [logits(rng, B, W, V) for _ in range(3)]
    ss = [beam_scores(rng, B, W) for _ in range(3)]
    x = torch.from_numpy(xs[0]).cuda()
    s = torch.from_numpy(ss[0].astype(np.float32)).cuda()
    out = (torch.empty(B, K, device="cuda"), torch.empty(B, K, dtype=torch.int32, device="cuda"),
           torch.empty(B, K, dtype=torch.int32, device="cuda"))
    assert mine.beam_select(x, s, K, out=out)[0] is out[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mine.beam_select(x, s, K, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mine.beam_select(x, s, K, out=out)
    mine.beam_select(torch.randn(8, 8, 40000, device="cuda"), torch.zeros(8, 8, device="cuda"), 32)
    for i in (1, 2):
        x.copy_(torch.from_numpy(xs[i]))
        s.copy_(torch.from_numpy(ss[i].astype(np.float32)))
        graph.replay()
        compare([host(a) for a in out], xs[i].astype(np.float64), ss[i].astype(np.float32).astype(np.float64), K)


def test_scores_in_place_and_stream_handles(torch_, ver):
    """The new scores may go where the old ones were (as many beams selected as
    there were); a stream may be given by its handle."""
    torch = torch_
    rng = np.random.default_rng(6)
    for B, W, V in ((3, 4, 500), (2, 9, 30000)):
        x, s = logits(rng, B, W, V), beam_scores(rng, B, W).astype(np.float32)
        t, old = torch.from_numpy(x).cuda(), torch.from_numpy(s).cuda()
        out = (old, torch.empty(B, W, dtype=torch.int32, device="cuda"), torch.empty(B, W, dtype=torch.int32, device="cuda"))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        ver.beam_select(t, old, W, out=out, stream=side.cuda_stream)
        compare([host(a) for a in out], x.astype(np.float64), s.astype(np.float64), W)


def test_many_requests(torch_, ver):
    """The largest batch, in one launch and in two."""
    torch = torch_
    g = torch.Generator("cuda")
    g.manual_seed(9)
    for W, V in ((2, 40), (20, 24)):
        x = torch.randn((65536, W, V), generator=g, device="cuda")
        s = -torch.rand((65536, W), generator=g, device="cuda")
        got = ver.beam_select(x, s, 2)
        c = (torch.log_softmax(x.double(), 2) + s.double()[..., None]).flatten(1)
        want, at = c.topk(2, 1)
        clear = (want[:, 0] - want[:, 1] > 8e-6) & (want[:, 1] - c.topk(3, 1).values[:, 2] > 8e-6)
        assert (got[0] - want).abs().max() < 4e-6 + 2.0**-24 * 20
        assert torch.equal(got[1][clear], (at // V).int()[clear]) and torch.equal(got[2][clear], (at % V).int()[clear])
        assert clear.float().mean() > 0.99
    with pytest.raises(Exception):
        ver.beam_select(torch.zeros(65537, 1, 4, device="cuda"), torch.zeros(65537, 1, device="cuda"), 1)


def test_shares_a_workspace_with_the_verifier(torch_, ver):
    """The top-8 thresholds that the verifier keeps in the workspace stay zero."""
    import gen
    import oracle
    from gpu_util import dev_i32, dev_logits
    rng = np.random.default_rng(2)
    inp = gen.greedy_synthetic(seed=5, B=8, k=4, V=5003, alpha=0.7, dtype="bf16")
    want = oracle.verify_greedy(inp.logits, inp.dtype, inp.drafts, topk=8)
    for _ in range(2):
        check(torch_, ver, logits(rng, 4, 8, 20000), beam_scores(rng, 4, 8), 32)
        got = [host(a) for a in ver.greedy(dev_logits(inp.logits, inp.dtype), dev_i32(inp.drafts), topk=8)]
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[2], want[2])


def test_refusals(torch_, ver):
    torch = torch_
    x, s = torch.zeros(2, 3, 64, device="cuda"), torch.zeros(2, 3, device="cuda")
    for call in (lambda: ver.beam_select(x, s.double(), 3), lambda: ver.beam_select(x, s[:, :2], 3),
                 lambda: ver.beam_select(x, s.t().contiguous().t(), 3), lambda: ver.beam_select(x[..., ::2], s, 3),
                 lambda: ver.beam_select(x, s, 3, finished=torch.zeros(2, 3, device="cuda")),
                 lambda: ver.beam_select(x, s, 3, out=(s, s, s))):
        with pytest.raises(ValueError):
            call()
    import speculative_decoding_draft_decode_b200 as sd
    for K in (0, 33):
        with pytest.raises(sd.SpecdecError):
            ver.beam_select(x, s, K)
    with pytest.raises(TypeError):
        ver.beam_select(x.half(), s, 3)
    assert ver.beam_select(x[:0], s[:0], 3)[0].shape == (0, 3)
