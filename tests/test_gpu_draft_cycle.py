"""The operators around the verify step in a run together, as a serving loop
uses them: the draft tree grown level by level by beam selection, the beams'
states carried along, slots planned, the tree verified, the accepted path's
states committed to the paged cache, over several steps and with requests that
end and start."""
import numpy as np
import pytest

import decode_reference as ref
import oracle
from gpu_util import host, require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_():
    return require_cuda()


V, D = 700, 24


def draft_row(token, position):
    """The toy draft model: logits of the next token."""
    rng = np.random.default_rng(1000003 * int(token) + int(position))
    x = rng.standard_normal(V).astype(np.float32) * 1.5
    x[(int(token) * 7 + 3) % V] += 6.0
    return x


def target_row(token, position):
    """The toy target model agrees with the draft's favourite most of the time."""
    x = draft_row(token, position).copy()
    if (int(token) + int(position)) % 4 == 0:
        x[(int(token) + 11) % V] += 20.0
    return x


def state_of(token, position, group):
    """What the cache holds for a token at a position."""
    return np.random.default_rng((int(token) * 131 + int(position)) * 7 + group).standard_normal(D).astype(np.float32)


def test_draft_verify_commit(torch_):
    import speculative_decoding_draft_decode_b200 as sd
    torch = torch_
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    ver = sd.Verifier(torch.device("cuda", 0))
    B, W, depth, G, bs, cols = 5, 4, 3, 2, 4, 16
    N = depth * W
    rng = np.random.default_rng(0)
    pages = B * cols
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    held = torch.zeros_like(lens)
    tables = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    ring = torch.arange(pages, dtype=torch.int32, device="cuda")
    ring_state = torch.tensor([0, pages], dtype=torch.int32, device="cuda")
    cache = torch.zeros(G, pages * bs, D, device="cuda")
    accept = torch.full((B,), -1, dtype=torch.int32, device="cuda")  # nothing to move on by yet
    texts = [[int(rng.integers(0, V))] for _ in range(B)]  # the last token's state is not in the cache yet
    for step in range(6):
        release = np.zeros(B, np.int32)
        if step == 3:  # two requests end, others take their places
            release[[1, 3]] = 1
            _, _, _, _, s = sd.plan_slots(lens, tables, held, ring, ring_state, bs, k=N, accept_len=accept,
                                          release=dev(release), out=(lens, held, ring_state,
                                                                     torch.empty(B * (N + 1), dtype=torch.int64, device="cuda"),
                                                                     torch.empty(B * (N + 1), dtype=torch.int64, device="cuda")))
            assert (host(lens)[[1, 3]] == 0).all() and (host(s).reshape(B, -1)[1] == -1).all()
            for b in (1, 3):
                texts[b] = [int(rng.integers(0, V))]
            accept = torch.full_like(accept, -1)  # the others have moved on in that call
        # grow the draft tree: W beams a level, their hidden states reordered with them
        parents = np.full((B, N + 1), -1, np.int32)
        tokens = np.full((B, N + 1), -1, np.int32)
        last = np.array([t[-1] for t in texts], np.int32)
        pos = np.array([len(t) - 1 for t in texts])
        beam_tok = np.repeat(last[:, None], W, 1)
        scores = np.full((B, W), -np.inf, np.float32)
        scores[:, 0] = 0.0
        nodes = np.zeros((B, W), np.int32)  # tree nodes of the beams
        hidden = dev(np.broadcast_to(last[None, :, None, None, None].astype(np.float32), (1, B, W, depth + 1, 8)).copy())
        for level in range(depth):
            x = np.stack([[draft_row(beam_tok[b, w], pos[b] + level) for w in range(W)] for b in range(B)])
            s, p, t = ver.beam_select(dev(x), dev(scores), W)
            sd.reorder_states(hidden, p)  # the beams' histories, in place
            hidden[0, :, :, level + 1] = t[..., None].float()
            e_s, e_p, e_t, _ = ref.beam_select(x.astype(np.float64), scores.astype(np.float64), W)
            s, p, t = host(s), host(p), host(t)
            assert np.array_equal(p, e_p) and np.array_equal(t, e_t) and np.allclose(s, e_s, atol=1e-5)
            first = 1 + level * W
            parents[:, first:first + W] = np.take_along_axis(nodes, p, 1)
            tokens[:, first:first + W] = t
            nodes = np.broadcast_to(np.arange(first, first + W, dtype=np.int32), (B, W))
            beam_tok, scores = t, s
        # every beam's carried history is its path in the tree
        got = host(hidden)[0, :, :, :, 0].astype(np.int32)
        for b in range(B):
            for w in range(W):
                path, c = [], nodes[b, w]
                while c > 0:
                    path.append(tokens[b, c])
                    c = parents[b, c]
                assert got[b, w].tolist() == [last[b]] + path[::-1]
        # slots of the N + 1 rows; the last step's accepted tokens are in the cache
        lens, held, ring_state, positions, slots = sd.plan_slots(lens, tables, held, ring, ring_state, bs, k=N,
                                                                 accept_len=accept)
        slots = slots.view(B, N + 1)
        assert np.array_equal(host(lens), [len(t) - 1 for t in texts]) and (host(slots) >= 0).all()
        # score the tree, verify it
        depth_of = np.zeros((B, N + 1), np.int64)
        for c in range(1, N + 1):
            depth_of[:, c] = np.take_along_axis(depth_of, parents[:, c:c + 1], 1)[:, 0] + 1
        tok_of = tokens.copy()
        tok_of[:, 0] = last
        x = np.stack([[target_row(tok_of[b, c], pos[b] + depth_of[b, c]) for c in range(N + 1)] for b in range(B)])
        al, acc_nodes, out = ver.tree(dev(x), dev(parents), dev(tokens), depth)
        want = oracle.verify_tree(x, "f32", parents, tokens, depth)
        assert all(np.array_equal(host(a), b) for a, b in zip((al, acc_nodes, out), want))
        # the tree's states to the cache, the accepted path only: from a buffer of their own, or in the cache itself
        src = np.stack([[[state_of(tok_of[b, c], pos[b] + depth_of[b, c], g) for c in range(N + 1)] for b in range(B)]
                        for g in range(G)])
        if step % 2:
            sd.commit_path(dev(src), al, acc_nodes, cache, slots)
        else:
            cache[:, slots] = dev(src)
            sd.commit_path(cache, al, acc_nodes, cache, slots, src_slots=slots)
        al_h, out_h = host(al), host(out)
        held_tokens = [t[:-1] + [t[-1]] + out_h[b, :al_h[b]].tolist() for b, t in enumerate(texts)]
        texts = [t + out_h[b, :al_h[b] + 1].tolist() for b, t in enumerate(texts)]
        # every position of every request holds its token's state
        tab, cch = host(tables), host(cache)
        for b, t in enumerate(held_tokens):
            for q, token in enumerate(t):
                slot = tab[b, q // bs] * bs + q % bs
                for g in range(G):
                    assert np.array_equal(cch[g, slot], state_of(token, q, g)), (step, b, q)
        accept = al
    assert sum(len(t) for t in texts) > 5 * 6  # drafts were accepted on the way
