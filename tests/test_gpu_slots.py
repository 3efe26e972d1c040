"""Block tables and slot maps on the GPU against the plain reference, exactly."""
import numpy as np
import pytest

import decode_reference as ref
from gpu_util import host, require_cuda

pytestmark = pytest.mark.gpu
FILL = -7


@pytest.fixture(scope="module")
def torch_():
    return require_cuda()


@pytest.fixture(scope="module")
def sd_(torch_):
    import speculative_decoding_draft_decode_b200 as sd
    return sd


def requests(rng, B, bs, cols, spare, max_len):
    lens = rng.integers(0, max_len + 1, B).astype(np.int32)
    held = np.minimum(-(-lens // bs) + rng.integers(0, 2, B), cols).astype(np.int32)
    pages = int(held.sum()) + spare
    perm = rng.permutation(pages).astype(np.int32)
    tables = np.full((B, cols), -1, np.int32)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    cap = pages + int(rng.integers(0, 5)) + 1
    head = int(rng.integers(0, cap))
    ring = np.full(cap, -99, np.int32)
    for i in range(spare):
        ring[(head + i) % cap] = perm[at + i]
    return lens, tables, held, ring, np.array([head, spare], np.int32)


def check(torch, sd, lens, tables, held, ring, state, bs, k=0, offsets=None, total=0, accept=None, release=None,
          in_place=False):
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    B = len(lens)
    rows = B * (k + 1) if offsets is None else B + total
    t_lens, t_tables, t_held, t_ring, t_state = dev(lens), dev(tables), dev(held), dev(ring), dev(state)
    pos = torch.full((rows,), FILL, dtype=torch.int64, device="cuda")
    slots = torch.full((rows,), FILL, dtype=torch.int64, device="cuda")
    if in_place:
        out = (t_lens, t_held, t_state, pos, slots)
    else:
        out = (torch.empty_like(t_lens), torch.empty_like(t_held), torch.empty_like(t_state), pos, slots)
    got = sd.plan_slots(t_lens, t_tables, t_held, t_ring, t_state, bs, k=k, draft_offsets=dev(offsets),
                        total_drafts=total, accept_len=dev(accept), release=dev(release), out=out)
    want = ref.plan_slots(lens, tables, held, ring, state, bs, k, offsets, total, accept, release, fill=FILL)
    for name, g, w in zip(("lens", "held", "state", "positions", "slots", "tables", "ring"), (*got, t_tables, t_ring), want):
        assert np.array_equal(host(g), w), name
    if not in_place:
        assert np.array_equal(host(t_lens), lens) and np.array_equal(host(t_held), held)
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,k,bs", [(1, 0, 1), (3, 4, 16), (64, 5, 16), (33, 64, 48), (500, 32, 8), (1024, 3, 64), (1025, 2, 16),
                                    (5000, 1, 16), (9000, 7, 4), (65536, 0, 16)])
def test_fixed_layout(torch_, sd_, B, k, bs, in_place):
    rng = np.random.default_rng(B + k)
    max_len = 300
    cols = (max_len + 2 * k + 2) // bs + 2
    lens, tables, held, ring, state = requests(rng, B, bs, cols, 2 * B * (k // bs + 2), max_len)
    accept = rng.integers(-1, k + 1, B).astype(np.int32)
    release = (rng.random(B) < 0.1).astype(np.int32)
    check(torch_, sd_, lens, tables, held, ring, state, bs, k, accept=accept, release=release, in_place=in_place)
    check(torch_, sd_, lens, tables, held, ring, state, bs, k)


@pytest.mark.parametrize("B", [1, 20, 1500, 8192, 8200])
def test_packed_layout(torch_, sd_, B):
    rng = np.random.default_rng(B)
    k, bs = 8, 16
    n = rng.integers(0, k + 1, B)
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    total = int(off[-1])
    lens, tables, held, ring, state = requests(rng, B, bs, 12, 3 * B, 100)
    accept = rng.integers(-1, k + 1, B).astype(np.int32)
    check(torch_, sd_, lens, tables, held, ring, state, bs, k, off, total, accept)
    # offsets that lie, run backwards or pass the total: those requests get nothing
    bad = off.copy()
    if B > 4:
        bad[3] = -1
        bad[9] = bad[8] - 1
        check(torch_, sd_, lens, tables, held, ring, state, bs, k, bad, total, accept)
        check(torch_, sd_, lens, tables, held, ring, state, bs, 3, off, min(total, 3 * B), accept)


def test_prompts(torch_, sd_):
    """Whole prompts: thousands of rows of a request, many pages each."""
    rng = np.random.default_rng(9)
    for bs in (1, 16, 100):
        n = np.array([0, 5000, 17, 1, 2500, 1024, 1023])
        B, k = len(n), 5000
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        lens, tables, held, ring, state = requests(rng, B, bs, 5200 // bs + 4, 12000 // bs + 20, 60)
        check(torch_, sd_, lens, tables, held, ring, state, bs, k, off, int(off[-1]))
    lens, tables, held, ring, state = requests(rng, 3, 32, 200, 400, 60)
    check(torch_, sd_, lens, tables, held, ring, state, 32, 4000)


@pytest.mark.parametrize("B", [40, 1300])
def test_too_few_pages(torch_, sd_, B):
    """The ring runs out part-way, is empty, or a table is full: those requests
    get no page, and rows without one get slot -1."""
    rng = np.random.default_rng(B)
    for spare in (0, 1, B // 2, B):
        for cols in (5, 30):
            lens, tables, held, ring, state = requests(rng, B, 4, cols, spare, 20)
            release = (rng.random(B) < 0.2).astype(np.int32)
            check(torch_, sd_, lens, tables, held, ring, state, 4, 9, release=release)


def test_bad_data(torch_, sd_):
    """Counts outside their ranges are clamped, negative pages map nowhere."""
    rng = np.random.default_rng(1)
    lens, tables, held, ring, state = requests(rng, 10, 8, 6, 30, 40)
    lens[0], held[1], held[2] = -5, -2, 99
    lens[3] = 2**31 - 1
    tables[4, 0] = -3
    check(torch_, sd_, lens, tables, held, ring, state, 8, 6, accept=np.full(10, 5, np.int32))


def test_far_slots(torch_, sd_):
    """Slots past 2^32: pages of 2^20 positions."""
    lens = np.array([3, 2**20 + 5], np.int32)
    tables = np.array([[9000, -1, -1], [2**31 - 1, 70000, -1]], np.int32)
    check(torch_, sd_, lens, tables, np.array([1, 2], np.int32), np.zeros(8, np.int32), np.array([0, 0], np.int32),
          2**20, 3)


def test_fresh_outputs_and_refusals(torch_, sd_):
    torch = torch_
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    side = torch.cuda.Stream()
    a = dict(seq_lens=i(2), block_tables=i(2, 4), held_blocks=i(2), free_ring=torch.arange(10, device="cuda").int(),
             ring_state=torch.tensor([0, 10], device="cuda").int(), block_size=16, k=3)
    side.wait_stream(torch.cuda.current_stream())
    lens, held, state, pos, slots = sd_.plan_slots(**a, stream=side)
    torch.cuda.synchronize()
    assert slots.tolist() == [0, 1, 2, 3, 16, 17, 18, 19] and state.tolist() == [2, 8] and held.tolist() == [1, 1]
    for bad in (dict(seq_lens=i(2).long()), dict(held_blocks=i(3)), dict(block_tables=i(3, 4)),
                dict(block_tables=i(4, 2).t()), dict(ring_state=i(3)), dict(free_ring=i(4, 2)), dict(accept_len=i(3)),
                dict(release=i(2).bool()), dict(draft_offsets=i(2)), dict(k=-2),
                dict(out=(i(2), i(2), i(2), i(8), i(8)))):
        with pytest.raises(ValueError):
            sd_.plan_slots(**{**a, **bad})
    for bad in (dict(block_size=0), dict(draft_offsets=i(3), total_drafts=9)):
        with pytest.raises(sd_.SpecdecError):
            sd_.plan_slots(**{**a, **bad})


def test_no_requests(torch_, sd_):
    """An empty batch leaves the ring as it was, in the outputs given too."""
    torch = torch_
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    pos, slots = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    state = torch.tensor([3, 7], device="cuda", dtype=torch.int32)
    a = (i(0), i(0, 4), i(0), i(10), state, 16)
    for kw in (dict(k=3), dict(k=3, draft_offsets=i(1))):
        out = (i(0), i(0), torch.full((2,), -9, device="cuda", dtype=torch.int32), pos, slots)
        assert sd_.plan_slots(*a, out=out, **kw)[2].tolist() == [3, 7]
        assert sd_.plan_slots(*a, **kw)[2].tolist() == [3, 7]
        assert sd_.plan_slots(*a, out=(i(0), i(0), state, pos, slots), **kw)[2].tolist() == [3, 7]


def test_uneven_rows(torch_, sd_):
    """Packed drafts that stand close together: one CTA's requests have most of
    the rows, more than it maps at a time."""
    rng = np.random.default_rng(21)
    for B in (1024, 3000):
        n = np.zeros(B, np.int64)
        n[5:505] = rng.integers(10, 32, 500)
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        lens, tables, held, ring, state = requests(rng, B, 16, 12, 3 * B, 100)
        check(torch_, sd_, lens, tables, held, ring, state, 16, 32, off, int(off[-1]))


@pytest.mark.parametrize("B", [50, 1500])
def test_steps_in_a_graph(torch_, sd_, B):
    """A decode loop's planning captured once and replayed: lengths, pages and
    the ring move on in place, step after step."""
    torch = torch_
    rng = np.random.default_rng(8)
    k, bs, cols = 4, 8, 40
    lens, tables, held, ring, state = requests(rng, B, bs, cols, 14 * B, 40)
    dev = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    t = dict(seq_lens=dev(lens), block_tables=dev(tables), held_blocks=dev(held), free_ring=dev(ring), ring_state=dev(state))
    accept, release = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    pos = torch.zeros(B * (k + 1), dtype=torch.int64, device="cuda")
    slots = torch.zeros_like(pos)
    call = lambda: sd_.plan_slots(**t, block_size=bs, k=k, accept_len=accept, release=release,  # noqa: E731
                                  out=(t["seq_lens"], t["held_blocks"], t["ring_state"], pos, slots))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(12):
        a = rng.integers(-1, k + 1, B).astype(np.int32)
        r = (rng.random(B) < 0.1).astype(np.int32)
        accept.copy_(torch.from_numpy(a))
        release.copy_(torch.from_numpy(r))
        graph.replay()
        lens, held, state, e_pos, e_slots, tables, ring = ref.plan_slots(lens, tables, held, ring, state, bs, k,
                                                                         accept=a, release=r)
        for g, w in ((t["seq_lens"], lens), (t["held_blocks"], held), (t["ring_state"], state), (pos, e_pos),
                     (slots, e_slots), (t["block_tables"], tables), (t["free_ring"], ring)):
            assert np.array_equal(host(g), w)
        used = e_slots[e_slots >= 0]
        assert len(set(used.tolist())) == len(used)
