"""Reordering of beam states and the commit of accepted paths: copies, so
every byte is compared."""
import numpy as np
import pytest

import decode_reference as ref
from gpu_util import host, require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_():
    return require_cuda()


@pytest.fixture(scope="module")
def sd_(torch_):
    import speculative_decoding_draft_decode_b200 as sd
    return sd


def bits(rng, shape, dtype):
    if dtype == "u8":
        return rng.integers(0, 256, shape).astype(np.uint8)
    if dtype == "i16":  # stands for bf16: the bits are moved
        return rng.integers(-30000, 30000, shape).astype(np.int16)
    return rng.standard_normal(shape).astype(np.float32)


def parents_of(rng, B, W, stray=True):
    p = rng.integers(0, W, (B, W)).astype(np.int32)
    if stray:
        p[rng.random((B, W)) < 0.15] = -1
        p[rng.random((B, W)) < 0.05] = W
    return p


@pytest.mark.parametrize("dtype", ["f32", "i16", "u8"])
@pytest.mark.parametrize("G,B,W,T,row", [(1, 1, 1, 1, (1,)), (2, 3, 2, 5, (8,)), (3, 2, 4, 33, (4, 16)), (2, 2, 5, 40, (7,)),
                                         (1, 3, 8, 300, (64,)), (2, 1, 16, 17, (24,)), (1, 2, 32, 50, (2, 20)),
                                         (1, 2, 9, 129, (250,)), (4, 1, 3, 2000, (1,))])
def test_reorder(torch_, sd_, dtype, G, B, W, T, row):
    torch = torch_
    rng = np.random.default_rng(G * 100 + W)
    for trial in range(3):
        src, old = bits(rng, (G, B, W, T, *row), dtype), bits(rng, (G, B, W, T, *row), dtype)
        par = parents_of(rng, B, W)
        lens = [None, rng.integers(0, T + 1, B).astype(np.int32),
                np.array([-3, T + 9, 1] * B, np.int32)[:B]][trial]
        p = torch.from_numpy(par).cuda()
        n = None if lens is None else torch.from_numpy(lens).cuda()
        x, to = torch.from_numpy(src).cuda(), torch.from_numpy(old).cuda()
        assert sd_.reorder_states(x, p, n, out=to) is to
        assert np.array_equal(host(to), ref.reorder_states(src, old, par, lens))
        assert np.array_equal(host(x), src)
        assert sd_.reorder_states(x, p, n) is x  # in place
        assert np.array_equal(host(x), ref.reorder_states(src, src, par, lens))


@pytest.mark.parametrize("W", [1, 3, 8, 20])
@pytest.mark.parametrize("D", [16, 33])
def test_reorder_heads_and_views(torch_, sd_, W, D):
    """Heads before positions, and views of a larger buffer whose other
    elements stay as they are."""
    torch = torch_
    rng = np.random.default_rng(W * D)
    G, B, H, T = 2, 3, 4, 21
    src, old = bits(rng, (G, B, W, H, T, D), "f32"), bits(rng, (G, B, W, H, T, D), "f32")
    par, lens = parents_of(rng, B, W), rng.integers(0, T + 1, B).astype(np.int32)
    p, n = torch.from_numpy(par).cuda(), torch.from_numpy(lens).cuda()
    want = ref.reorder_states(src, old, par, lens, time_dim=4)
    to = torch.from_numpy(old).cuda()
    sd_.reorder_states(torch.from_numpy(src).cuda(), p, n, time_dim=4, out=to)
    assert np.array_equal(host(to), want)
    # positions of a larger cache, a part of each row, requests in another order of memory
    big = torch.full((B, G, W, H, T + 3, D + 5), -1.0, device="cuda")
    view = big[:, :, :, :, 1:T + 1, 2:D + 2].permute(1, 0, 2, 3, 4, 5)
    view.copy_(torch.from_numpy(src))
    keep = host(big).copy()
    sd_.reorder_states(view, p, n, time_dim=4)
    full = keep.copy()
    full[:, :, :, :, 1:T + 1, 2:D + 2] = ref.reorder_states(src, src, par, lens, 4).transpose(1, 0, 2, 3, 4, 5)
    assert np.array_equal(host(big), full)


def test_reorder_far_strides(torch_, sd_):
    """Byte offsets past 2^32: two groups 5 GB apart, beams 1 GB apart."""
    torch = torch_
    buf = torch.empty(10_000_000_000, dtype=torch.uint8, device="cuda")
    x = torch.as_strided(buf, (2, 1, 3, 10, 64), (5_000_000_000, 4_000_000_000, 1_000_000_000, 64, 1))
    rng = np.random.default_rng(0)
    src = bits(rng, (2, 1, 3, 10, 64), "u8")
    x.copy_(torch.from_numpy(src))
    par = np.array([[2, 0, 0]], np.int32)
    sd_.reorder_states(x, torch.from_numpy(par).cuda())
    assert np.array_equal(host(x), ref.reorder_states(src, src, par, None))


@pytest.mark.parametrize("T,D", [(29, 33), (200, 7), (9, 255), (16, 8)])
@pytest.mark.parametrize("first,gap", [(0, 0), (1, 0), (3, 5), (7, 16)])
def test_reorder_odd_runs(torch_, sd_, T, D, first, gap):
    """2-byte rows of odd size at odd addresses, out of place: every phase of a
    beam's run against 16 bytes, with the bytes around the runs left alone."""
    torch = torch_
    rng = np.random.default_rng(T + first)
    G, B, W = 2, 3, 7
    run = T * D + gap
    n = first + G * B * W * run + 40

    def view(buf):
        return torch.as_strided(buf, (G, B, W, T, D), (B * W * run, W * run, run, D, 1), first)

    src = torch.from_numpy(rng.integers(-30000, 30000, n).astype(np.int16)).cuda()
    dst = torch.from_numpy(rng.integers(-30000, 30000, n).astype(np.int16)).cuda()
    par, lens = parents_of(rng, B, W), np.array([T, T // 2, 1], np.int32)
    old, flat = host(view(dst)).copy(), host(dst).copy()
    sd_.reorder_states(view(src), torch.from_numpy(par).cuda(), torch.from_numpy(lens).cuda(), out=view(dst))
    want = ref.reorder_states(host(view(src)), old, par, lens)
    assert np.array_equal(host(view(dst)), want)
    again = torch.from_numpy(flat).cuda()
    view(again).copy_(torch.from_numpy(want))
    assert np.array_equal(host(dst), host(again))


def test_reorder_many_items(torch_, sd_):
    """More work items than resident CTAs, ragged: every item is taken."""
    torch = torch_
    g = torch.Generator("cuda")
    g.manual_seed(3)
    x = torch.randint(0, 30000, (40, 32, 4, 70, 96), generator=g, device="cuda", dtype=torch.int16)
    old = torch.zeros_like(x)
    rng = np.random.default_rng(4)
    par, lens = parents_of(rng, 32, 4, stray=False), rng.integers(0, 71, 32).astype(np.int32)
    got = sd_.reorder_states(x, torch.from_numpy(par).cuda(), torch.from_numpy(lens).cuda(), out=old)
    assert np.array_equal(host(got), ref.reorder_states(host(x), np.zeros(x.shape, np.int16), par, lens))


@pytest.mark.parametrize("shape", [(70000, 1, 2, 3, 4), (1, 65536, 2, 2, 2), (3, 2, 5, 11)])
def test_reorder_large_counts(torch_, sd_, shape):
    """More groups or requests than a grid has rows; token histories (a position
    is one element)."""
    torch = torch_
    rng = np.random.default_rng(shape[1])
    src, old = bits(rng, shape, "f32"), bits(rng, shape, "f32")
    par = parents_of(rng, shape[1], shape[2])
    x, to = torch.from_numpy(src).cuda(), torch.from_numpy(old).cuda()
    sd_.reorder_states(x, torch.from_numpy(par).cuda(), out=to)
    ok = (par >= 0) & (par < shape[2])
    idx = np.where(ok, par, 0)
    moved = src[:, np.arange(shape[1])[:, None], idx]
    keep = ok.reshape(1, *par.shape, *([1] * (len(shape) - 3)))
    assert np.array_equal(host(to), np.where(keep, moved, old))
    sd_.reorder_states(x, torch.from_numpy(par).cuda())
    assert np.array_equal(host(x), np.where(keep, moved, src))


def test_reorder_graph_and_stream(torch_, sd_):
    torch = torch_
    rng = np.random.default_rng(6)
    src = bits(rng, (2, 2, 4, 9, 16), "f32")
    x, p = torch.from_numpy(src).cuda(), torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    to = torch.zeros_like(x)
    side.wait_stream(torch.cuda.current_stream())
    sd_.reorder_states(x, p, out=to, stream=side)
    torch.cuda.synchronize()
    assert np.array_equal(host(to), np.repeat(src[:, :, :1], 4, 2))
    with torch.cuda.graph(graph):
        sd_.reorder_states(x, p)
    for i in range(2):
        par = parents_of(rng, 2, 4)
        p.copy_(torch.from_numpy(par))
        src = ref.reorder_states(src, src, par, None)
        graph.replay()
        assert np.array_equal(host(x), src)


def test_reorder_refusals(torch_, sd_):
    torch = torch_
    x = torch.zeros(2, 3, 4, 5, 6, device="cuda")
    p = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    big = torch.zeros(3, 3, 4, 5, 6, device="cuda")
    for call in (lambda: sd_.reorder_states(x, p.long()), lambda: sd_.reorder_states(x, p[:2]),
                 lambda: sd_.reorder_states(x, p, n[:2]), lambda: sd_.reorder_states(x, p, n.float()),
                 lambda: sd_.reorder_states(x, p, out=x[:1]), lambda: sd_.reorder_states(x, p, out=x.half()),
                 lambda: sd_.reorder_states(big[:2], p, out=big[1:]),
                 lambda: sd_.reorder_states(x[..., ::2], p), lambda: sd_.reorder_states(x, p, time_dim=2),
                 lambda: sd_.reorder_states(x[..., 0], p, time_dim=4),
                 lambda: sd_.reorder_states(x, p, out=x[:, :1].expand(2, 3, 4, 5, 6).clone()[:, :, :1].expand(2, 3, 4, 5, 6))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sd_.SpecdecError):
        sd_.reorder_states(torch.zeros(1, 1, 33, 2, 4, device="cuda"), torch.zeros(1, 33, dtype=torch.int32, device="cuda"))
    assert sd_.reorder_states(x[:, :0], p[:0]).shape[1] == 0


def paths(rng, B, N, depth):
    """Accepted lengths and ascending node indices, as tree verification returns them."""
    al = rng.integers(-1, min(depth, N) + 1, B).astype(np.int32)
    nodes = np.full((B, depth), -1, np.int32)
    for b in range(B):
        if al[b] > 0:
            nodes[b, :al[b]] = np.sort(rng.choice(N, al[b], replace=False)) + 1
    return al, nodes


@pytest.mark.parametrize("dtype", ["f32", "i16", "u8"])
@pytest.mark.parametrize("G,B,N,depth,row", [(1, 1, 0, 1, (1,)), (2, 3, 5, 4, (8,)), (3, 16, 64, 6, (2, 64)), (1, 4, 40, 32, (33,)),
                                             (2, 2, 100, 9, (1000,)), (2, 5, 12, 12, (4096,))])
def test_commit(torch_, sd_, dtype, G, B, N, depth, row):
    torch = torch_
    rng = np.random.default_rng(N + depth)
    src = bits(rng, (G, B, N + 1, *row), dtype)
    S = B * (depth + 3) + 5
    old = bits(rng, (G, S, *row), dtype)
    al, nodes = paths(rng, B, N, depth)
    slots = rng.permutation(S)[:B * (depth + 2)].reshape(B, depth + 2).astype(np.int64)
    slots[rng.random(slots.shape) < 0.05] = -1
    slots[rng.random(slots.shape) < 0.02] = S
    if B > 2:
        nodes[2, 0] = N + 1   # no such node
        al[2] = max(al[2], 1)
        al[1] = depth + 4     # past the table: clamped
        nodes[1] = np.sort(rng.choice(N, depth, replace=N < depth)) + 1
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    to = dev(old)
    assert sd_.commit_path(dev(src), dev(al), dev(nodes), to, dev(slots)) is to
    assert np.array_equal(host(to), ref.commit_path(src, al, nodes, old, slots))


@pytest.mark.parametrize("N,depth,row", [(8, 4, 16), (64, 6, 256), (200, 32, 40), (40, 20, 7)])
def test_commit_in_place(torch_, sd_, N, depth, row):
    """The tree was scored in the cache itself: node c in the slot of position len + c."""
    torch = torch_
    rng = np.random.default_rng(N)
    G, B = 3, 7
    S = B * (N + 1) + 11
    cache = bits(rng, (G, S, row), "f32")
    slots = rng.permutation(S)[:B * (N + 1)].reshape(B, N + 1).astype(np.int64)
    al, nodes = paths(rng, B, N, depth)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    x, sl = dev(cache), dev(slots)
    sd_.commit_path(x, dev(al), dev(nodes), x, sl, src_slots=sl)
    assert np.array_equal(host(x), ref.commit_path(cache, al, nodes, cache, slots, slots))
    # from another cache, by its own slots
    y, z = dev(cache), dev(bits(rng, (G, S + 3, row), "f32"))
    want = ref.commit_path(cache, al, nodes, host(z), slots + 2, slots)
    sd_.commit_path(y, dev(al), dev(nodes), z, dev(slots + 2), src_slots=sl)
    assert np.array_equal(host(z), want) and np.array_equal(host(y), cache)


@pytest.mark.parametrize("G,B", [(70000, 1), (1, 65536)])
def test_commit_large_counts(torch_, sd_, G, B):
    torch = torch_
    rng = np.random.default_rng(G)
    src, cache = bits(rng, (G, B, 3, 2), "f32"), bits(rng, (G, 2 * B + 3, 2), "f32")
    al = rng.integers(-1, 2, B).astype(np.int32)
    nodes = rng.integers(1, 3, (B, 1)).astype(np.int32)
    slots = rng.permutation(2 * B + 3)[:2 * B].reshape(B, 2).astype(np.int64)
    to = torch.from_numpy(cache.copy()).cuda()
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    sd_.commit_path(dev(src), dev(al), dev(nodes), to, dev(slots))
    want = cache.copy()
    b = np.nonzero(al >= 0)[0]
    want[:, slots[b, 0]] = src[:, b, 0]
    b = np.nonzero(al >= 1)[0]
    want[:, slots[b, 1]] = src[:, b, nodes[b, 0]]
    assert np.array_equal(host(to), want)


def test_commit_refusals(torch_, sd_):
    torch = torch_
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    src, dst = torch.zeros(2, 3, 5, 8, device="cuda"), torch.zeros(2, 40, 8, device="cuda")
    sl = torch.zeros(3, 5, dtype=torch.int64, device="cuda")
    ok = lambda **k: sd_.commit_path(**{**dict(src=src, accept_len=i(3), accept_nodes=i(3, 4), dst=dst, dst_slots=sl), **k})  # noqa: E731
    ok()
    for bad in (dict(accept_len=i(2)), dict(accept_len=i(3).long()), dict(accept_nodes=i(3)), dict(dst=dst.half()),
                dict(dst_slots=sl[:, :4]), dict(dst_slots=sl.int()), dict(dst_slots=sl[:2]), dict(dst=dst[:1]),
                dict(src=src[:, :2]), dict(src=src[..., :4]), dict(src=dst), dict(dst=src.view(2, 15, 8)),
                dict(src=dst, src_slots=sl.int()), dict(src=dst[:, 1:], dst=dst[:, :39], src_slots=sl),
                dict(src=src[..., ::2], dst=dst[..., ::2])):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(sd_.SpecdecError):
        sd_.commit_path(src, i(3), i(3, 33), dst, torch.zeros(3, 34, dtype=torch.int64, device="cuda"))


def test_rows_that_share_memory(torch_, sd_):
    """Windows of one buffer: a row written is a part of another one."""
    torch = torch_
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    flat = torch.zeros(4096, device="cuda")
    for shape, strides in (((1, 2, 3, 4, 8), (0, 96, 8, 8, 1)), ((2, 2, 3, 4, 8), (64, 96, 32, 8, 1)),
                           ((1, 2, 3, 4, 8), (0, 88, 32, 8, 1))):
        x = flat.as_strided(shape, strides)
        with pytest.raises(ValueError, match="share memory"):
            sd_.reorder_states(x, i(*shape[1:3]))
        with pytest.raises(ValueError, match="share memory"):
            sd_.reorder_states(torch.zeros(shape, device="cuda"), i(*shape[1:3]), out=x)
    sl = torch.zeros(3, 5, dtype=torch.int64, device="cuda")
    for strides in ((8, 8, 1), (16, 12, 1), (72, 8, 1)):
        with pytest.raises(ValueError, match="share memory"):
            sd_.commit_path(torch.zeros(2, 3, 5, 8, device="cuda"), i(3), i(3, 4), flat.as_strided((2, 10, 8), strides), sl)
    # groups within positions, and gaps anywhere, are no such case
    for t in (flat[:2 * 10 * 8].view(10, 2, 8).transpose(0, 1), flat.as_strided((2, 10, 8), (11, 30, 1))):
        sd_.commit_path(torch.zeros(2, 3, 5, 8, device="cuda"), i(3) - 1, i(3, 4), t, sl)
    x = torch.zeros(4, 3, 2, 5, 8, device="cuda").permute(2, 1, 3, 0, 4)
    assert sd_.reorder_states(x, i(3, 5)) is x


def test_other_current_device_is_refused(torch_, sd_, monkeypatch):
    """Tensors of another device than the current one: refused, nothing launched."""
    torch = torch_
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    x, p = torch.zeros(1, 2, 3, 4, 5, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError, match="current device"):
        sd_.reorder_states(x, p)
    with pytest.raises(ValueError, match="current device"):
        sd_.commit_path(torch.zeros(1, 2, 3, 4, device="cuda"), i(2), i(2, 2), torch.zeros(1, 9, 4, device="cuda"),
                        torch.zeros(2, 3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="current device"):
        sd_.plan_slots(i(2), i(2, 4), i(2), i(10), i(2), 16, out=(i(2), i(2), i(2), i(2).long(), i(2).long()))
    with pytest.raises(ValueError):
        sd_.Verifier(torch.device("cuda", 0)).beam_select(x[0, 0].contiguous(), torch.zeros(3, 4, device="cuda"), 2)
