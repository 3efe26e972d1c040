"""Host-side checks of the operators around the verify step: every refusal
comes before any CUDA call, so these run without a GPU."""
import os
import subprocess
import sys

import pytest
import torch

import speculative_decoding_draft_decode_b200 as sd
from speculative_decoding_draft_decode_b200 import build as sd_build

FAKE = 0x7F0000000000  # never dereferenced: every case below fails its checks first
E, U, W, OK = sd.SPECDEC_ERR_INVALID_ARG, sd.SPECDEC_ERR_UNSUPPORTED, sd.SPECDEC_ERR_WORKSPACE, sd.SPECDEC_OK


@pytest.fixture(scope="module", autouse=True)
def built():
    sd_build.build()


def beam(**kw):
    a = dict(logits=FAKE, dtype=0, row_stride=1000, beam_scores=FAKE, finished=None, eos_token=0, B=4, W=4, K=4,
             V=1000, out_scores=FAKE, out_parents=FAKE, out_tokens=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=0)
    a.update(kw)
    return sd.specdec_beam_select(**a)


def test_beam_refusals():
    assert beam(dtype=5) == U
    for bad in (dict(B=-1), dict(B=sd.MAX_B + 1), dict(W=0), dict(W=33), dict(K=0), dict(K=33), dict(V=0),
                dict(V=(1 << 24) + 1), dict(row_stride=999), dict(logits=None), dict(beam_scores=None),
                dict(out_scores=None), dict(out_parents=None), dict(out_tokens=None), dict(logits=FAKE + 2),
                dict(finished=FAKE, eos_token=1000), dict(finished=FAKE, eos_token=-1)):
        assert beam(**bad) == E, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 4), dict(ws_bytes=1024)):
        assert beam(**bad) == W, bad
    assert beam(B=0, logits=None) == OK


def test_beam_workspace_size():
    f = sd.specdec_workspace_size_beam
    assert f(64, 8, 8, 128256, sd.SPECDEC_BF16) > 65536 * 4
    assert f(64, 16, 8, 128256, sd.SPECDEC_BF16) > f(64, 8, 8, 128256, sd.SPECDEC_BF16)
    assert f(0, 8, 8, 1000, 0) >= 65536 * 4
    for bad in ((-1, 4, 4, 100, 0), (4, 0, 4, 100, 0), (4, 33, 4, 100, 0), (4, 4, 0, 100, 0), (4, 4, 33, 100, 0),
                (4, 4, 4, 0, 0), (4, 4, 4, 100, 2)):
        assert f(*bad) == 0, bad
    # a larger batch, more beams or a longer row never needs less
    for small, large in (((7, 8, 4, 70000, 1), (8, 8, 4, 70000, 1)), ((3, 10, 4, 128256, 0), (4, 10, 4, 128256, 0)),
                         ((4, 8, 4, 128000, 1), (4, 9, 4, 128000, 1)), ((63, 4, 4, 16000, 0), (64, 4, 4, 16000, 0)),
                         ((16, 8, 4, 31000, 1), (16, 8, 4, 33000, 1))):
        assert f(*small) <= f(*large)
    need = f(4, 4, 4, 1000, 0)
    assert beam(ws_bytes=need - 1) == W


def reorder(**kw):
    a = dict(src=FAKE, dst=FAKE + (1 << 30), parents=FAKE, lengths=None, G=2, B=2, W=4, H=1, T=8, row_bytes=64,
             src_strides=(4096, 2048, 512, 0, 64), dst_strides=(4096, 2048, 512, 0, 64), stream=0)
    a.update(kw)
    return sd.specdec_reorder_states(**a)


def test_reorder_refusals():
    for bad in (dict(B=-1), dict(B=sd.MAX_B + 1), dict(W=0), dict(W=33), dict(G=-1), dict(H=-1), dict(T=-1),
                dict(row_bytes=-1), dict(src=None), dict(dst=None), dict(parents=None), dict(T=1 << 41),
                dict(T=1 << 40, row_bytes=1 << 40), dict(src_strides=(-1, 2048, 512, 0, 64)),
                dict(dst=FAKE, dst_strides=(4096, 2048, 512, 0, 128))):
        assert reorder(**bad) == E, bad
    for none in (dict(B=0), dict(G=0), dict(H=0), dict(T=0), dict(row_bytes=0)):
        assert reorder(src=None, **none) == OK


def commit(**kw):
    a = dict(src=FAKE, src_group_stride=1 << 20, src_request_stride=1 << 12, src_row_stride=64, src_slots=None,
             src_slots_stride=0, src_rows=0, dst=FAKE + (1 << 32), dst_group_stride=1 << 20, dst_row_stride=64,
             dst_slots=FAKE, dst_slots_stride=7, dst_rows=100, accept_len=FAKE, accept_nodes=FAKE, G=2, B=2, N=10,
             max_depth=6, row_bytes=64, stream=0)
    a.update(kw)
    return sd.specdec_commit_path(**a)


def test_commit_refusals():
    for bad in (dict(B=-1), dict(N=-1), dict(N=1024), dict(max_depth=0), dict(max_depth=33), dict(G=-1),
                dict(row_bytes=-1), dict(dst_slots_stride=6), dict(src_slots=FAKE, src_slots_stride=10),
                dict(src_row_stride=63), dict(dst_row_stride=63), dict(src=None), dict(dst=None),
                dict(dst_slots=None), dict(accept_len=None), dict(accept_nodes=None), dict(src_rows=-1),
                dict(dst_rows=-1), dict(src_group_stride=-1), dict(G=1 << 40, row_bytes=1 << 40)):
        assert commit(**bad) == E, bad
    for none in (dict(B=0), dict(G=0), dict(row_bytes=0)):
        assert commit(src=None, **none) == OK


def plan(**kw):
    a = dict(seq_lens=FAKE, accept_len=None, release=None, draft_offsets=None, B=4, k=4, total_drafts=0,
             block_size=16, block_tables=FAKE, table_stride=8, max_blocks=8, held_blocks=FAKE, free_ring=FAKE,
             ring_capacity=100, ring_state=FAKE, seq_lens_out=FAKE, held_out=FAKE, ring_state_out=FAKE,
             positions=FAKE, slots=FAKE, stream=0)
    a.update(kw)
    return sd.specdec_plan_slots(**a)


def test_plan_refusals():
    for bad in (dict(B=-1), dict(B=sd.MAX_B + 1), dict(k=-1), dict(k=sd.MAX_PLAN_ROWS), dict(block_size=0),
                dict(block_size=sd.MAX_PLAN_ROWS + 1), dict(max_blocks=0), dict(table_stride=7),
                dict(ring_capacity=0), dict(draft_offsets=FAKE, total_drafts=-1),
                dict(draft_offsets=FAKE, total_drafts=17), dict(seq_lens=None), dict(block_tables=None),
                dict(held_blocks=None), dict(free_ring=None), dict(ring_state=None), dict(seq_lens_out=None),
                dict(held_out=None), dict(ring_state_out=None), dict(positions=None), dict(slots=None)):
        assert plan(**bad) == E, bad
    assert plan(B=0, seq_lens=None) == OK


def apart(*names):
    return {n: FAKE + (i << 32) for i, n in enumerate(names)}


def test_beam_outputs_that_share_memory():
    """An output over another one, or over an input that other requests still
    read; only the scores may take the old ones' place, as many as they are."""
    a = dict(apart("logits", "beam_scores", "out_scores", "out_parents", "out_tokens", "ws", "finished"), K=8)
    for bad in (dict(out_scores=a["beam_scores"]), dict(out_parents=a["out_scores"]), dict(out_tokens=a["out_parents"] + 124),
                dict(out_scores=a["beam_scores"] + 60), dict(out_scores=a["beam_scores"] + 4, K=4),
                dict(out_tokens=a["finished"]), dict(out_parents=a["beam_scores"], K=4),
                dict(out_scores=a["logits"] + 15 * 4000 + 3996), dict(out_parents=a["ws"] + 1024),
                dict(out_parents=a["finished"], K=4)):
        assert beam(**{**a, **bad}) == E, bad


def test_plan_outputs_that_share_memory():
    a = apart("seq_lens", "accept_len", "release", "draft_offsets", "block_tables", "held_blocks", "free_ring",
              "ring_state", "seq_lens_out", "held_out", "ring_state_out", "positions", "slots")
    a["total_drafts"] = 16
    for bad in (dict(seq_lens_out=a["held_out"]), dict(seq_lens_out=a["held_blocks"]), dict(held_out=a["seq_lens"]),
                dict(held_out=a["held_blocks"] + 4), dict(ring_state_out=a["ring_state"] + 4),
                dict(ring_state_out=a["free_ring"] + 396), dict(positions=a["slots"]), dict(slots=a["positions"] + 152),
                dict(slots=a["draft_offsets"] + 16), dict(positions=a["accept_len"]), dict(seq_lens_out=a["release"]),
                dict(block_tables=a["free_ring"]), dict(block_tables=a["seq_lens"] - 124), dict(free_ring=a["held_blocks"])):
        assert plan(**{**a, **bad}) == E, bad


def test_host_tensors_are_refused():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ver = sd.Verifier(torch.device("cuda", 0))
    with pytest.raises(ValueError):
        ver.beam_select(torch.zeros(2, 3, 64), torch.zeros(2, 3), 3)
    with pytest.raises(ValueError):
        sd.reorder_states(torch.zeros(1, 2, 3, 4, 5), i(2, 3))
    with pytest.raises(ValueError):
        sd.commit_path(torch.zeros(1, 2, 3, 4), i(2), i(2, 2), torch.zeros(1, 9, 4), torch.zeros(2, 3).long())
    with pytest.raises(ValueError):
        sd.plan_slots(i(2), i(2, 4), i(2), i(10), i(2), 16, k=3)


class OnGpu1:
    """Stands for a tensor of another GPU."""
    device = torch.device("cuda", 1)
    is_cuda = True

    def numel(self):
        return 2


def test_other_streams_are_refused(monkeypatch):
    """A stream of another device than the current one is refused before the
    native code sees anything."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = OnGpu1()

    class Here(OnGpu1):
        device = torch.device("cuda", 0)

    for args in (dict(stream=x), dict(stream=OnGpu1())):
        for t in (x, Here()):
            with pytest.raises(ValueError, match="current device"):
                sd.Verifier(torch.device("cuda", 0)).beam_select(t, t, 3, **args)
            with pytest.raises(ValueError, match="current device"):
                sd.reorder_states(t, t, **args)
            with pytest.raises(ValueError, match="current device"):
                sd.commit_path(t, t, t, t, t, **args)
            with pytest.raises(ValueError, match="current device"):
                sd.plan_slots(t, t, t, t, t, 16, **args)


def test_binding_refuses_what_is_no_tensor():
    b = sd._bind()
    with pytest.raises(TypeError):
        b.reorder_states([1], None, None, 3, None, None, 0)
    with pytest.raises(TypeError):
        b.reorder_states()
    with pytest.raises(TypeError):
        b.plan_slots(*[None] * 14)
    with pytest.raises(OverflowError):
        b.commit_path(*[torch.zeros(1)] * 6, None, 1 << 80)
    with pytest.raises(ValueError, match="CUDA device tensors"):
        b.reorder_states(torch.zeros(1, 1, 1, 1, 4), torch.zeros(1, 1).int(), None, 3, None, None, 0)


def test_outgrown_workspaces_are_kept(monkeypatch):
    """A captured graph holds the workspace's address: growing the workspace
    for a larger call must not free the smaller one."""
    monkeypatch.setattr(sd, "specdec_workspace_init", lambda ws, n, stream=None: sd.SPECDEC_OK)
    ver = sd.Verifier(torch.device("cpu"))
    first, n = ver.workspace(1000)
    ver.workspace(5000)
    assert ver._ws is not first and any(w is first for w in ver._outgrown)


def test_binding_loads_before_torch_is_imported():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = "import speculative_decoding_draft_decode_b200 as sd; sd._bind()"
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_the_library_is_built_without_torch(monkeypatch, tmp_path, capsys):
    """C programs use the library alone: a machine without PyTorch builds it."""
    monkeypatch.setattr(sd_build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setitem(sys.modules, "torch", None)
    assert sd_build.build() == sd_build.LIB
    assert not (tmp_path / "_binding.so").exists() and "not built" in capsys.readouterr().err


def test_a_binding_of_another_torch_is_stale(monkeypatch):
    import importlib.metadata
    assert sd_build.up_to_date()
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.1")
    assert not sd_build.up_to_date()
