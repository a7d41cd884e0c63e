"""What the linear attention, beam selection and reordering entry points refuse, before anything
is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import ssd_sequence_mixing_b200 as ssd

FAKE = 1 << 20  # an aligned, never-dereferenced device address
F = ctypes.c_void_p(FAKE)
ODD = ctypes.c_void_p(FAKE + 4)
lib = ssd.library()


def shape(**kw):
    d = dict(batch=2, seqlen=300, nheads=4, headdim=64, dstate=128, ngroups=2, nseq=0, io_dtype=ssd.SSD_BF16, cu=None)
    d.update(kw)
    return ssd.SsdShape(d["batch"], d["seqlen"], d["nheads"], d["headdim"], d["dstate"], d["ngroups"], d["nseq"],
                        d["io_dtype"], d["cu"])


def forward(s, cu=None, per_token=1, **p):
    a = {n: F for n in ("q", "k", "v", "log_decay", "y")}
    a.update(p)
    g = lambda n: a.get(n)
    return lib.ssd_linear_attention_forward(s and ctypes.byref(s), g("q"), g("k"), g("v"), g("log_decay"), per_token, 1.0,
                                            g("init"), cu, g("y"), g("final"), None)


def backward(s, cu=None, per_token=1, **p):
    a = {n: F for n in ("dy", "q", "k", "v", "log_decay", "dq", "dk", "dv")}
    a.update(p)
    g = lambda n: a.get(n)
    return lib.ssd_linear_attention_backward(s and ctypes.byref(s), g("dy"), g("q"), g("k"), g("v"), g("log_decay"),
                                             per_token, 1.0, g("init"), g("dfinal"), cu, g("dq"), g("dk"), g("dv"),
                                             g("dlog"), g("dinit"), None)


def step(s, **p):
    a = {n: F for n in ("q", "k", "v", "log_decay", "state", "y")}
    a.update(p)
    g = lambda n: a.get(n)
    return lib.ssd_linear_attention_step(s and ctypes.byref(s), g("q"), g("k"), g("v"), g("log_decay"), 1, 1.0,
                                         g("state"), g("y"), None)


@pytest.mark.parametrize("call", [forward, backward, lambda s, **k: step(s, **k)], ids=["forward", "backward", "step"])
def test_shapes(call):
    one = dict(seqlen=1) if call not in (forward, backward) else {}
    assert call(None) == 1
    for kw in (dict(batch=-1), dict(nheads=0), dict(headdim=0), dict(dstate=0), dict(ngroups=0), dict(io_dtype=7)):
        assert call(shape(**{**one, **kw})) == 1, kw
    for kw in (dict(headdim=129), dict(dstate=129), dict(nheads=6, ngroups=4), dict(nheads=70000, ngroups=1),
               dict(batch=1 << 31)):
        assert call(shape(**{**one, **kw})) == 2, kw


@pytest.mark.parametrize("call,names", [(forward, ("q", "k", "v", "log_decay", "y")),
                                        (backward, ("dy", "q", "k", "v", "log_decay", "dq", "dk", "dv")),
                                        (lambda s, **k: step(s, **k), ("q", "k", "v", "log_decay", "state", "y"))],
                         ids=["forward", "backward", "step"])
def test_pointers(call, names):
    s = shape() if call in (forward, backward) else shape(seqlen=1)
    for n in names:
        assert call(s, **{n: None}) == 1, n
        assert call(s, **{n: ODD}) == 3, n
    optional = {forward: ("init", "final"), backward: ("init", "dfinal", "dlog", "dinit")}.get(call, ())
    for n in optional:
        assert call(s, **{n: ODD}) == 3, n


def test_packed_batches():
    for call in (forward, backward):
        assert call(shape(batch=2, nseq=3), cu=F) == 1
        assert call(shape(batch=1, nseq=0), cu=F) == 1
        assert call(shape(batch=1, nseq=2), cu=ODD) == 3
        for vals in ([1, 5, 300], [0, 5, 299], [0, 400, 300]):
            host = torch.tensor(vals, dtype=torch.int32)
            assert call(shape(batch=1, nseq=2, cu=host.data_ptr()), cu=F) == 6
        # the grid's limit
        assert call(shape(batch=1, seqlen=1 << 29, nheads=4096, nseq=1), cu=F) == 2


def test_nothing_to_do():
    assert forward(shape(batch=0), q=None, k=None, v=None, y=None, log_decay=None) == 0
    assert backward(shape(batch=0), dy=None, q=None, k=None, v=None, log_decay=None, dq=None, dk=None, dv=None) == 0
    assert step(shape(batch=0, seqlen=1)) == 0
    assert step(shape(seqlen=2)) == 1


def select(batch=2, beams=4, vocab=100, dtype=ssd.SSD_F32, eos=-1, count=4, **p):
    a = {n: F for n in ("logits", "scores", "s", "t", "p")}
    a.update(p)
    g = lambda n: a.get(n)
    return lib.ssd_beam_select(batch, beams, vocab, dtype, g("logits"), g("scores"), g("finished"), eos, count, g("s"),
                               g("t"), g("p"), None)


def test_select():
    for kw in (dict(batch=-1), dict(beams=0), dict(vocab=0), dict(count=0), dict(dtype=5), dict(finished=F, eos=-1),
               dict(finished=F, eos=100), dict(logits=None), dict(scores=None), dict(s=None), dict(t=None), dict(p=None)):
        assert select(**kw) == 1, kw
    for kw in (dict(beams=65), dict(count=65), dict(vocab=(1 << 20) + 1), dict(batch=1 << 25)):
        assert select(**kw) == 2, kw
    for n in ("logits", "scores", "finished", "s", "t", "p"):
        assert select(**{n: ODD, "eos": 1}) == 3, n
    assert select(batch=0, logits=None) == 0


def reorder(batch=2, beams=4, parents=F, bufs=(FAKE,), sizes=(64,), n=None):
    b = (ctypes.c_void_p * max(1, len(bufs)))(*bufs)
    s = (ctypes.c_int64 * max(1, len(sizes)))(*sizes)
    return lib.ssd_state_reorder(batch, beams, parents, len(bufs) if n is None else n, b, s, None)


def test_reorder():
    assert reorder(batch=-1) == 1
    assert reorder(beams=0) == 1
    assert reorder(n=-1) == 1
    assert reorder(beams=65) == 2
    assert reorder(parents=None) == 1
    assert reorder(parents=ctypes.c_void_p(FAKE + 2)) == 3
    assert reorder(bufs=(None,)) == 1
    assert reorder(bufs=(FAKE + 8,)) == 3
    assert reorder(sizes=(-1,)) == 1
    assert reorder(sizes=(1 << 40,)) == 2
    assert reorder(bufs=(FAKE, FAKE), sizes=(64, 64)) == 1  # the same rows twice
    assert reorder(bufs=(FAKE + 256, FAKE), sizes=(64, 64)) == 1  # 8 rows of 64 bytes reach into the other
    assert reorder(batch=0) == 0
    assert reorder(bufs=()) == 0
    assert lib.ssd_linear_attention_forward(None, *([None] * 4), 1, 1.0, *([None] * 5)) == 1


def test_binding_checks():
    """The binding's own checks, on host tensors: the device first, then shapes and types."""
    x = torch.zeros(1, 4, 2, 8)
    for f in (lambda: ssd.linear_attention_forward(x, x, x, torch.zeros(2)),
              lambda: ssd.linear_attention_backward(x, x, x, x, torch.zeros(2)),
              lambda: ssd.linear_attention_step(x[0], x[0], x[0], torch.zeros(2), torch.zeros(4, 2, 8, 8)),
              lambda: ssd.beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2)),
              lambda: ssd.state_reorder(x, torch.zeros(1, 1, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            f()
